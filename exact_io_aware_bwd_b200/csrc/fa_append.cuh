// Append of new keys and values to a paged key/value cache, with the position
// rotation of keys and queries applied on the way.
//
// Token t of sequence b (n new tokens, L cached tokens with them) sits at
// position p = L - n + t, slot p % P of physical page table[b][p / P].  Its
// feature pairs (x, y) of the first rot features are turned by the angle
// a_i = p * inv_freq[i]:
//   x' = x cos a_i - y sin a_i,   y' = x sin a_i + y cos a_i
// pair i being features (i, i + rot/2), or (2i, 2i + 1) when interleaved;
// the other features, and v, are copied.
//
// The angle of a far position has no fraction left in 32 bits (p = 10^6 times
// 1.0 keeps 4 bits of it), so turns = p * inv_freq / (2 pi) is formed in 64
// bits, its whole part dropped there, and only the remaining fraction of a
// turn rounded to 32 bits (error below 2^-25 turns).  Products and sums are in
// 32 bits and rounded once to the I/O type.
//
// A thread owns one (token, slot), a slot being 16 features of a row (two
// 16-byte vectors: the two halves of 8 pairs, or 16 neighbouring features when
// interleaved), and walks over heads: its 8 sines and cosines are computed
// once and serve every query and key head.
//
// Bound by memory on prompts: 16 384 tokens of 32 / 8 heads of 128 (436 MB read
// and written) in 72 us, 6.0 TB/s; by the launch on single tokens, 2.9 us.
// Several heads' loads in flight a thread (78 us against 112 with one), three
// resident blocks (80 registers, 24 to 32 bytes of spills) and 24 blocks per
// SM (72 us against 78 with 4) got it there; ragged batches stay at the latency
// of their first loads.
#pragma once

#include <type_traits>

#include "fa_decode.cuh"  // programmatic dependent launch, kStatusBadInput

namespace fa {

constexpr uint32_t kKernAppend = 15;
constexpr int kAppendThreads = 256;
// Heads whose loads a thread has in flight (2, or 3 at four resident blocks:
// 83-85 us on the prompt above against 80).
constexpr int kAppendHeads = 4;

struct AppendParams {
  const void* q;  // nullptr: keys and values only
  const void* k;
  const void* v;
  // strides in elements: batch, head, token
  long long qs[3], ks[3], vs[3];
  void* q_out;    // [B][Hq][N][d]
  void* k_out;    // [B][Hkv][N][d] or nullptr
  void* k_cache;  // [num_pages][Hkv][P][d]
  void* v_cache;
  const int* table;     // [B][max_pages]
  const int* lens;      // [B]
  const int* new_lens;  // [B] or nullptr: N each
  const float* inv_freq;  // [rot / 2]
  long long tokens;       // B * N
  int Hq, Hkv, N, d, P, max_pages, num_pages, rot;
  int tok_per_block;      // threads: tok_per_block * d / 16 * head lanes
};

// 1 / (2 pi)
constexpr double kInvTwoPi = 0.15915494309189533576888;

template <bool BF16, bool INTER>
__global__ void __launch_bounds__(kAppendThreads, 3) fa_append_kernel(const __grid_constant__ AppendParams p) {
  using T = typename std::conditional<BF16, __nv_bfloat16, __half>::type;
  using T2 = typename std::conditional<BF16, __nv_bfloat162, __half2>::type;
  grid_dependency_wait();
  grid_launch_dependents();
  const int slots = p.d / 16;
  const int s = threadIdx.x % slots;
  const int row = threadIdx.x / slots;
  const int head_lanes = kAppendThreads / (slots * p.tok_per_block);
  const long long tok = static_cast<long long>(blockIdx.x) * p.tok_per_block + row % p.tok_per_block;
  if (tok >= p.tokens) return;
  const int b = static_cast<int>(tok / p.N), t = static_cast<int>(tok % p.N);
  const int L = p.lens[b];
  if (L == 0) return;  // idle sequence
  const int n = p.new_lens ? p.new_lens[b] : p.N;
  if (n < 0 || n > p.N || L < n || L > static_cast<long long>(p.max_pages) * p.P) {
    if (t == 0 && s == 0) record_error(kStatusBadInput, kKernAppend, 0, 0);
    return;
  }
  if (t >= n) return;
  const int pos = L - n + t;
  const int phys = p.table[static_cast<size_t>(b) * p.max_pages + pos / p.P];
  const bool page_ok = phys >= 0 && phys < p.num_pages;
  if (!page_ok && s == 0) record_error(kStatusBadInput, kKernAppend, 0, 1);

  // the slot's two vectors (first feature of each) and its first pair
  const int half = p.rot / 2;
  const bool turned = INTER ? 16 * s < p.rot : 8 * s < half;
  const int c0 = INTER || !turned ? 16 * s : 8 * s;
  const int c1 = INTER || !turned ? c0 + 8 : c0 + half;

  const T* q = static_cast<const T*>(p.q) + b * p.qs[0] + t * p.qs[2];
  const T* k = static_cast<const T*>(p.k) + b * p.ks[0] + t * p.ks[2];
  const T* v = static_cast<const T*>(p.v) + b * p.vs[0] + t * p.vs[2];
  const int Hq = p.q ? p.Hq : 0;
  const int heads = Hq + 2 * p.Hkv;  // query heads, then key heads, then value heads
  const int step = gridDim.y * head_lanes;
  int h = blockIdx.y * head_lanes + row / p.tok_per_block;
  auto load = [&](int hh, uint4& a, uint4& c) {
    if (hh >= heads) return;
    const T* src = hh < Hq ? q + hh * p.qs[1] : hh < Hq + p.Hkv ? k + (hh - Hq) * p.ks[1] : v + (hh - Hq - p.Hkv) * p.vs[1];
    a = *reinterpret_cast<const uint4*>(src + c0);
    c = *reinterpret_cast<const uint4*>(src + c1);
  };
  // kAppendHeads heads in flight at a time; the first ones are asked for
  // before the sines and cosines are computed
  uint4 a[kAppendHeads], c[kAppendHeads];
#pragma unroll
  for (int u = 0; u < kAppendHeads; ++u) load(h + u * step, a[u], c[u]);

  float cs[8], sn[8];
  if (turned) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const double turns = static_cast<double>(pos) * (static_cast<double>(p.inv_freq[8 * s + i]) * kInvTwoPi);
      sincospif(2.f * static_cast<float>(turns - rint(turns)), &sn[i], &cs[i]);
    }
  }
  auto turn = [&](uint4& av, uint4& cv) {
    const T2* a2 = reinterpret_cast<const T2*>(&av);
    const T2* c2 = reinterpret_cast<const T2*>(&cv);
    float x[8], y[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      // half split: a holds the x of pairs 2i, 2i + 1, c their y;
      // interleaved: a holds pair i, c pair 4 + i
      const float2 u = make_float2(static_cast<float>(a2[i].x), static_cast<float>(a2[i].y));
      const float2 w = make_float2(static_cast<float>(c2[i].x), static_cast<float>(c2[i].y));
      if (INTER) {
        x[i] = u.x, y[i] = u.y, x[4 + i] = w.x, y[4 + i] = w.y;
      } else {
        x[2 * i] = u.x, x[2 * i + 1] = u.y, y[2 * i] = w.x, y[2 * i + 1] = w.y;
      }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float xi = x[i], yi = y[i];
      x[i] = xi * cs[i] - yi * sn[i];
      y[i] = xi * sn[i] + yi * cs[i];
    }
    uint32_t aw[4], cw[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      aw[i] = INTER ? pack2<BF16>(x[i], y[i]) : pack2<BF16>(x[2 * i], x[2 * i + 1]);
      cw[i] = INTER ? pack2<BF16>(x[4 + i], y[4 + i]) : pack2<BF16>(y[2 * i], y[2 * i + 1]);
    }
    av = make_uint4(aw[0], aw[1], aw[2], aw[3]);
    cv = make_uint4(cw[0], cw[1], cw[2], cw[3]);
  };
  // this token's rows of head 0; a head further is N (outputs) or P (cache) rows
  const long long slot = static_cast<long long>(phys) * p.Hkv * p.P + pos % p.P;
  T* q_out = static_cast<T*>(p.q_out) + (static_cast<long long>(b) * p.Hq * p.N + t) * p.d;
  T* k_out = static_cast<T*>(p.k_out) + (static_cast<long long>(b) * p.Hkv * p.N + t) * p.d;
  auto put = [&](T* dst, const uint4& av, const uint4& cv) {
    *reinterpret_cast<uint4*>(dst + c0) = av;
    *reinterpret_cast<uint4*>(dst + c1) = cv;
  };
  auto store = [&](int hh, uint4& av, uint4& cv) {
    if (hh >= heads) return;
    if (turned && hh < Hq + p.Hkv) turn(av, cv);
    if (hh < Hq) {
      put(q_out + static_cast<long long>(hh) * p.N * p.d, av, cv);
    } else if (hh < Hq + p.Hkv) {
      const long long g = hh - Hq;
      if (page_ok) put(static_cast<T*>(p.k_cache) + (slot + g * p.P) * p.d, av, cv);
      if (p.k_out) put(k_out + g * p.N * p.d, av, cv);
    } else if (page_ok) {
      put(static_cast<T*>(p.v_cache) + (slot + static_cast<long long>(hh - Hq - p.Hkv) * p.P) * p.d, av, cv);
    }
  };
  for (;;) {
#pragma unroll
    for (int u = 0; u < kAppendHeads; ++u) store(h + u * step, a[u], c[u]);
    h += kAppendHeads * step;
    if (h >= heads) break;
#pragma unroll
    for (int u = 0; u < kAppendHeads; ++u) load(h + u * step, a[u], c[u]);
  }
}

}  // namespace fa
