// The second half of decode behind a shared prefix: every sequence's own keys
// (those behind the prefix), joined with the prefix's partial results that
// fa_paged_kernel left in the workspace.
//
// A block takes the R = G Nq <= 32 rows of one (sequence, kv head).  Each
// cached byte is used once, for R rows, so the work is bound by memory and,
// sequences' own parts being short, by latency: the fragments of the products
// (16 rows x 16 keys) are loaded from the cache straight into registers, with
// no staging and no barrier until the block's end.  The order of a product's
// inner index is free, so the features of Q and K are dealt to the lanes in
// 16-byte pieces: the 4 lanes of a key read 64 neighbouring bytes.  For P V the
// lane's 4 keys are read 16 bytes at a time, the 8 lanes of a key 128
// neighbouring bytes, and neighbouring keys paired by byte permutes.  (tcgen05
// needs 128 keys staged in shared memory and takes its result through tensor
// memory: the decode kernel built on it needs about 4 us for a sequence
// of 150 keys however few they are; here a group of 16 keys is 32 small MMAs.)
//
// Warps take groups of 16 keys in turn (with more than 16 rows, two warps per
// group, one for each 16 rows), each with its own running max and sum; K of
// the next group is in flight during P V of this one, V during its scores.
// The partial results of the warps and of the prefix's splits meet at the end:
//   m* = max m_s, l* = sum l_s 2^(m_s - m*), O = sum O_s 2^(m_s - m*) / l*.
// With few sequences the own keys are split over several blocks, and
// fa_paged_merge_kernel joins them instead.
#pragma once

#include "fa_paged.cuh"

namespace fa {

constexpr uint32_t kKernPrefixOwn = 14;
constexpr int kOwnWarps = 4;
constexpr int kOwnThreads = 32 * kOwnWarps;

struct OwnParams {
  PagedParams p;        // the prefix pass: sizes, its partial results, o, lse
  const void* q;        // [B][Hq][N][d]
  const void* k_cache;  // [num_pages][Hkv][P][d]
  const void* v_cache;
  float* own_o;         // [row][S][d], [row][S][2]: with S > 1
  float* own_ml;
  int S;
  int follows;          // the prefix kernel precedes this one in the stream
};

template <bool BF16>
__device__ __forceinline__ void mma_16816(float* c, const uint32_t* a, uint32_t b0, uint32_t b1) {
  if constexpr (BF16)
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Shared memory: the warps' O [warp][16][d] and (m, l) [warp][16].
template <int HD>
constexpr int own_smem() { return kOwnWarps * 16 * (HD * 4 + 8); }

// WM: warps that share a group of keys, one for each 16 rows.
template <int HD, bool BF16, int WM>
__global__ void __launch_bounds__(kOwnThreads, HD == 128 ? 2 : 4) fa_prefix_own_kernel(const __grid_constant__ OwnParams a) {
  using T = typename std::conditional<BF16, __nv_bfloat16, __half>::type;
  const PagedParams& p = a.p;
  constexpr int kC = HD / 32;   // 16-byte pieces of a lane's K (or Q) row
  constexpr int kH = HD / 64;   // 128-byte pieces of a V row
  constexpr int kW = kOwnWarps / WM;  // warps along the keys
  extern __shared__ float4 own_sm[];
  float* sO = reinterpret_cast<float*>(own_sm);
  float2* sML = reinterpret_cast<float2*>(sO + kOwnWarps * 16 * HD);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int nn = lane >> 2, qd = lane & 3;
  const int kw = warp / WM, mt = warp % WM;
  const int split = blockIdx.x % a.S, item = blockIdx.x / a.S;
  const int b = item / p.Hkv, g = item % p.Hkv;
  const int R = p.G * p.N;

  // The inputs were written before the prefix kernel started (it waits for
  // them before it lets this kernel be scheduled); only its results are
  // waited for, at the end.
  if (!a.follows) grid_dependency_wait();
  grid_launch_dependents();

  const int L = p.lens[b];
  const bool bad = L != 0 && (L < p.N || L > static_cast<long long>(p.max_pages) * p.P);
  if (bad && g == 0 && split == 0 && threadIdx.x == 0) record_error(kStatusBadInput, kKernPrefixOwn, 0, 0);
  // groups of 16 keys: of the sequence's own part, and of this split
  const int own = bad || L <= p.prefix ? 0 : L - p.prefix;
  const int n_groups = (own + 15) / 16;
  const int g0 = static_cast<int>(static_cast<long long>(n_groups) * split / a.S);
  const int g1 = static_cast<int>(static_cast<long long>(n_groups) * (split + 1) / a.S);

  // Q: rows mt * 16 + nn and + 8 as the A operand
  const T* q = static_cast<const T*>(a.q) + (static_cast<size_t>(b) * p.Hkv + g) * R * HD;
  uint32_t qa[kC][2][4];
  int lim[2];  // last key the two rows see
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const int r = mt * 16 + nn + 8 * e;
    lim[e] = L - p.N + r % p.N;
#pragma unroll
    for (int c = 0; c < kC; ++c) {
      uint4 w = make_uint4(0u, 0u, 0u, 0u);
      if (r < R) w = *reinterpret_cast<const uint4*>(q + static_cast<size_t>(r) * HD + c * 32 + qd * 8);
      qa[c][0][e] = w.x, qa[c][0][e + 2] = w.y, qa[c][1][e] = w.z, qa[c][1][e + 2] = w.w;
    }
  }

  float o[8 * kH][4];
#pragma unroll
  for (int j = 0; j < 8 * kH; ++j)
#pragma unroll
    for (int e = 0; e < 4; ++e) o[j][e] = 0.f;
  float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};

  const int* row = p.table + static_cast<size_t>(b) * p.max_pages;
  // element offset of key 0 of group gi in the caches, -1: nothing to load
  auto group_base = [&](int gi) -> long long {
    if (gi >= g1) return -1;
    const int key = p.prefix + 16 * gi;
    const int phys = __ldg(row + key / p.P);
    if (phys < 0 || phys >= p.num_pages) {
      if (lane == 0) record_error(kStatusBadInput, kKernPrefixOwn, 0, 1);
      return -1;
    }
    return ((static_cast<long long>(phys) * p.Hkv + g) * p.P + key % p.P) * HD;
  };
  const T* kc = static_cast<const T*>(a.k_cache);
  const T* vc = static_cast<const T*>(a.v_cache);
  uint4 kf[2][kC], vf[4][kH];
  // slots without a token are not read: zeros
  auto load_k = [&](int gi, long long base) {
    const int left = L - p.prefix - 16 * gi;  // keys from the group's first on
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int c = 0; c < kC; ++c) {
        kf[j][c] = make_uint4(0u, 0u, 0u, 0u);
        if (base >= 0 && 8 * j + nn < left)
          kf[j][c] = *reinterpret_cast<const uint4*>(kc + base + (8 * j + nn) * HD + c * 32 + qd * 8);
      }
  };
  auto load_v = [&](int gi, long long base) {
    const int left = L - p.prefix - 16 * gi;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int key = 2 * qd + (e & 1) + 8 * (e >> 1);
#pragma unroll
      for (int c = 0; c < kH; ++c) {
        vf[e][c] = make_uint4(0u, 0u, 0u, 0u);
        if (base >= 0 && key < left) vf[e][c] = *reinterpret_cast<const uint4*>(vc + base + key * HD + c * 64 + nn * 8);
      }
    }
  };

  int gi = g0 + kw;
  long long base = group_base(gi), base_next = group_base(gi + kW);
  load_k(gi, base);
  load_v(gi, base);
  for (; gi < g1; gi += kW) {
    float s[2][4];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      s[j][0] = s[j][1] = s[j][2] = s[j][3] = 0.f;
#pragma unroll
      for (int c = 0; c < kC; ++c) {
        mma_16816<BF16>(s[j], qa[c][0], kf[j][c].x, kf[j][c].y);
        mma_16816<BF16>(s[j], qa[c][1], kf[j][c].z, kf[j][c].w);
      }
    }
    base = base_next;
    base_next = group_base(gi + 2 * kW);
    load_k(gi + kW, base);
    // scores in log2 units, hidden keys -inf: element 2e + x is row e
    const int key0 = p.prefix + 16 * gi + 2 * qd;
    float mx[2] = {m[0], m[1]};
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float v = s[j][e] * p.scale_log2;
        s[j][e] = key0 + 8 * j + (e & 1) <= lim[e >> 1] ? v : -INFINITY;
        mx[e >> 1] = fmaxf(mx[e >> 1], s[j][e]);
      }
    float fac[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      mx[e] = fmaxf(mx[e], __shfl_xor_sync(0xffffffffu, mx[e], 1));
      mx[e] = fmaxf(mx[e], __shfl_xor_sync(0xffffffffu, mx[e], 2));
      fac[e] = mx[e] == -INFINITY ? 1.f : ex2_approx(m[e] - mx[e]);
    }
    const bool moves = mx[0] > m[0] || mx[1] > m[1];
    if (__any_sync(0xffffffffu, moves)) {
#pragma unroll
      for (int j = 0; j < 8 * kH; ++j) {
        o[j][0] *= fac[0], o[j][1] *= fac[0];
        o[j][2] *= fac[1], o[j][3] *= fac[1];
      }
      l[0] *= fac[0], l[1] *= fac[1];
      m[0] = mx[0], m[1] = mx[1];
    }
    const float ref[2] = {m[0] == -INFINITY ? 0.f : m[0], m[1] == -INFINITY ? 0.f : m[1]};
    uint32_t pa[4];
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float x = ex2_approx(s[j][2 * e] - ref[e]), y = ex2_approx(s[j][2 * e + 1] - ref[e]);
        l[e] += x + y;
        pa[2 * j + e] = pack2<BF16>(x, y);
      }
#pragma unroll
    for (int c = 0; c < kH; ++c) {
      const uint32_t* v0 = reinterpret_cast<const uint32_t*>(&vf[0][c]);
      const uint32_t* v1 = reinterpret_cast<const uint32_t*>(&vf[1][c]);
      const uint32_t* v2 = reinterpret_cast<const uint32_t*>(&vf[2][c]);
      const uint32_t* v3 = reinterpret_cast<const uint32_t*>(&vf[3][c]);
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        mma_16816<BF16>(o[8 * c + 2 * w], pa, __byte_perm(v0[w], v1[w], 0x5410), __byte_perm(v2[w], v3[w], 0x5410));
        mma_16816<BF16>(o[8 * c + 2 * w + 1], pa, __byte_perm(v0[w], v1[w], 0x7632), __byte_perm(v2[w], v3[w], 0x7632));
      }
    }
    load_v(gi + kW, base);
  }

  // The warp's rows into shared memory: lane holds features c 64 + qd 16 + i
  // (element 0 of o[8 c + i]; + 8: element 1) of rows nn (and + 8: 2, 3).
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    l[e] += __shfl_xor_sync(0xffffffffu, l[e], 1);
    l[e] += __shfl_xor_sync(0xffffffffu, l[e], 2);
    const int r = warp * 16 + nn + 8 * e;
    if (qd == 0) sML[r] = make_float2(m[e], l[e]);
    if (mt * 16 + nn + 8 * e < R)
#pragma unroll
      for (int c = 0; c < kH; ++c)
#pragma unroll
        for (int x = 0; x < 2; ++x)
#pragma unroll
          for (int i = 0; i < 8; i += 4)
            *reinterpret_cast<float4*>(sO + r * HD + c * 64 + qd * 16 + 8 * x + i) =
                make_float4(o[8 * c + i][2 * e + x], o[8 * c + i + 1][2 * e + x], o[8 * c + i + 2][2 * e + x],
                            o[8 * c + i + 3][2 * e + x]);
  }
  if (a.S == 1 && a.follows) grid_dependency_wait();  // the prefix's partial results
  __syncthreads();
  const bool last = a.S == 1;
  const int tile = b / p.seqs;
  const bool single = (p.n_tiles & 1) && tile == p.n_tiles - 1;
  const int slots = last ? (single ? p.S_single : p.S) : 0;  // 0 without a prefix
  const long long part = (static_cast<long long>(g) * p.n_tiles + tile) * p.slots;
  for (int x = threadIdx.x; x < R * (HD / 4); x += kOwnThreads) {
    const int r = x / (HD / 4), c4 = x % (HD / 4);
    const int hg = r / p.N, t = r % p.N;
    const int tr = ((b % p.seqs) * p.N + t) * p.G + hg;  // row of the prefix's tile: (sequence, token, head)
    const float2* ml = p.part_ml + part * 128 + tr;
    const float4* po = p.part_o + (part * (HD / 4) + c4) * 128 + tr;
    float ms = -INFINITY;
#pragma unroll
    for (int w = 0; w < kW; ++w) ms = fmaxf(ms, sML[(w * WM + r / 16) * 16 + r % 16].x);
#pragma unroll 8
    for (int s = 0; s < slots; ++s) ms = fmaxf(ms, ml[s * 128].x);
    float ls = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    auto add = [&](float2 y, const float4* src) {
      if (y.x == -INFINITY) return;
      const float w = ex2_approx(y.x - ms);
      const float4 z = *src;
      ls += y.y * w;
      acc.x += z.x * w, acc.y += z.y * w, acc.z += z.z * w, acc.w += z.w * w;
    };
#pragma unroll
    for (int w = 0; w < kW; ++w) {
      const int sr = (w * WM + r / 16) * 16 + r % 16;
      add(sML[sr], reinterpret_cast<const float4*>(sO + sr * HD) + c4);
    }
#pragma unroll 4
    for (int s = 0; s < slots; ++s) add(ml[s * 128], po + static_cast<long long>(s) * (HD / 4) * 128);
    const long long out = (static_cast<long long>(b) * p.Hkv + g) * R + r;
    if (last) {
      const float inv = ls > 0.f ? 1.f / ls : 0.f;
      uint2 w;
      w.x = pack2<BF16>(acc.x * inv, acc.y * inv);
      w.y = pack2<BF16>(acc.z * inv, acc.w * inv);
      *reinterpret_cast<uint2*>(static_cast<T*>(p.o) + out * HD + 4 * c4) = w;
      if (c4 == 0) p.lse[out] = ls > 0.f ? (ms + __log2f(ls)) * 0.69314718055994531f : -INFINITY;
    } else {
      reinterpret_cast<float4*>(a.own_o + (out * a.S + split) * HD)[c4] = acc;
      if (c4 == 0) reinterpret_cast<float2*>(a.own_ml)[out * a.S + split] = make_float2(ms, ls);
    }
  }
  // the prefix kernel, too, is complete before this one is: whoever waits for
  // this kernel may read what both left
  if (a.S > 1 && a.follows) grid_dependency_wait();
}

}  // namespace fa
