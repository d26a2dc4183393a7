// Whether two strided tensors share memory: what a call's outputs must not do with its inputs (host code).
#pragma once

#include <cstdint>
#include <initializer_list>
#include <numeric>

namespace moe {

// T tokens' rows of H heads, `width` bytes each; strides in bytes, not negative, not used for one token or one head.
struct Rows {
  uintptr_t at;
  long long T, token, H, head, width;
};

inline Rows whole(const void* p, long long bytes) { return {reinterpret_cast<uintptr_t>(p), 1, 0, 1, 0, bytes}; }

// False where rows share memory, and also where the ranges of addresses overlap and the token strides of several tokens differ.
inline bool rows_apart(Rows a, Rows b) {
  if (a.T < 1 || a.H < 1 || b.T < 1 || b.H < 1 || a.width < 1 || b.width < 1) return true;
  for (Rows* r : {&a, &b}) {
    if (r->T == 1) r->token = 0;
    if (r->H == 1) r->head = 0;
  }
  const long long tokens_a = (a.T - 1) * a.token, tokens_b = (b.T - 1) * b.token;
  const long long heads_a = (a.H - 1) * a.head, heads_b = (b.H - 1) * b.head;
  if (a.at + tokens_a + heads_a + a.width <= b.at || b.at + tokens_b + heads_b + b.width <= a.at) return true;
  if (a.T > 1 && b.T > 1 && a.token != b.token) return false;
  const long long token = a.T > 1 ? a.token : b.token, d0 = static_cast<long long>(b.at) - static_cast<long long>(a.at);
  // Side by side in every period: of a token, of a head, of the largest step that all strides are multiples of.
  auto beside = [d0](long long period, long long wa, long long wb) {
    if (period < 1) return false;
    const long long r = ((d0 % period) + period) % period;
    return r >= wa && r + wb <= period;
  };
  if (beside(token, heads_a + a.width, heads_b + b.width)) return true;
  if ((a.H == 1 || b.H == 1 || a.head == b.head) && beside(a.H > 1 ? a.head : b.head, tokens_a + a.width, tokens_b + b.width)) return true;
  if (beside(std::gcd(token, std::gcd(a.head, b.head)), a.width, b.width)) return true;
  // Head by head: rows t2 of b and t1 of a lie d + (t2 - t1) * token bytes apart.
  auto floor_div = [](long long x, long long y) { return x / y - (x % y != 0 && x < 0); };
  for (long long i = 0; i < a.H; ++i) {
    for (long long j = 0; j < b.H; ++j) {
      const long long d = d0 + j * b.head - i * a.head;
      if (token == 0) {
        if (d < a.width && -d < b.width) return false;
        continue;
      }
      // -b.width < d + m token < a.width
      const long long least = floor_div(-b.width - d, token) + 1, most = floor_div(a.width - d - 1, token);
      if ((least > 1 - a.T ? least : 1 - a.T) <= (most < b.T - 1 ? most : b.T - 1)) return false;
    }
  }
  return true;
}

}  // namespace moe
