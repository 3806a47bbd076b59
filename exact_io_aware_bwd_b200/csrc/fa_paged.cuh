// Attention of rows of new tokens over a paged key/value cache: the forward
// pass of many new tokens (fa_fwd_paged) and decode of a batch that shares a
// prefix (fa_decode_prefix).  One warp per query row, one key at a time.
#pragma once

#include <type_traits>

#include "fa_decode.cuh"  // programmatic dependent launch, kStatusBadInput

namespace fa {

constexpr uint32_t kKernPaged = 13;

struct PagedParams {
  const void* q;
  const void* k_cache;
  const void* v_cache;
  const int* table;
  const int* lens;
  const int* new_lens;
  void* o;
  float* lse;
  long long rows;
  int Hq, Hkv, N, P, max_pages, num_pages;
  int prefix;  // keys below it: the pages of sequence 0
  float scale_log2;
};

template <int HD, bool BF16>
__global__ void __launch_bounds__(256) fa_paged_rows_kernel(const __grid_constant__ PagedParams p) {
  using T = typename std::conditional<BF16, __nv_bfloat16, __half>::type;
  constexpr int E = HD / 32;
  const int lane = threadIdx.x & 31;
  const long long row = static_cast<long long>(blockIdx.x) * 8 + (threadIdx.x >> 5);
  if (row >= p.rows) return;
  const int t = static_cast<int>(row % p.N);
  const int h = static_cast<int>(row / p.N % p.Hq), b = static_cast<int>(row / p.N / p.Hq);
  const int g = h / (p.Hq / p.Hkv);
  const int L = p.lens[b];
  const int n = p.new_lens ? p.new_lens[b] : p.N;
  const bool bad = n < 0 || n > p.N || L < n || L > static_cast<long long>(p.max_pages) * p.P;
  if (L != 0 && bad && h == 0 && t == 0 && lane == 0) record_error(kStatusBadInput, kKernPaged, 0, 0);
  if (p.new_lens && !bad && t >= n) return;
  const T* q = static_cast<const T*>(p.q) + row * HD;
  float qv[E], acc[E], m = -INFINITY, l = 0.f;
  for (int e = 0; e < E; ++e) {
    qv[e] = static_cast<float>(q[lane * E + e]);
    acc[e] = 0.f;
  }
  const int last = L == 0 || bad ? -1 : L - n + t;
  for (int key = 0; key <= last; ++key) {
    const int phys = p.table[(key < p.prefix ? 0 : static_cast<size_t>(b) * p.max_pages) + key / p.P];
    if (phys < 0 || phys >= p.num_pages) {
      if (lane == 0) record_error(kStatusBadInput, kKernPaged, 0, 1);
      continue;
    }
    const long long off = ((static_cast<long long>(phys) * p.Hkv + g) * p.P + key % p.P) * HD + lane * E;
    const T* k = static_cast<const T*>(p.k_cache) + off;
    const T* v = static_cast<const T*>(p.v_cache) + off;
    float s = 0.f;
    for (int e = 0; e < E; ++e) s += qv[e] * static_cast<float>(k[e]);
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    s *= p.scale_log2;
    const float mn = fmaxf(m, s);
    const float w = exp2f(m - mn), x = exp2f(s - mn);
    m = mn;
    l = l * w + x;
    for (int e = 0; e < E; ++e) acc[e] = acc[e] * w + x * static_cast<float>(v[e]);
  }
  T* o = static_cast<T*>(p.o) + row * HD;
  for (int e = 0; e < E; ++e) o[lane * E + e] = static_cast<T>(l > 0.f ? acc[e] / l : 0.f);
  if (lane == 0) p.lse[row] = l > 0.f ? (m + log2f(l)) * 0.69314718055994531f : -INFINITY;
}

}  // namespace fa
