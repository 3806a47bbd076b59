// The second half of decode behind a shared prefix: every sequence's own keys
// (those behind the prefix), joined with the prefix's partial results that
// fa_paged_kernel left in the workspace.
//
// A block takes the R = G Nq <= 32 rows of one (sequence, kv head).  Each
// cached byte is used once, for R rows, so the work is bound by memory and,
// sequences' own parts being short, by latency.  A warp therefore runs its
// own ring of two stages (K and V rows of 16 keys at d = 128, 32 at d = 64, as
// TMA boxes of 16 rows x 128 bytes), with no barrier between warps until
// the end, and 16 x 16 fragments go from shared memory to mma.sync: 16 rows
// are one of its tiles, and a group of 16 keys 32 of its instructions.
// (tcgen05 takes 128 rows or keys at a time and its result through tensor
// memory: the decode kernel built on it needs about 4 us for a sequence of 150
// keys however few its rows are.)
// The order of a product's inner index is free, so the features of Q and K
// are dealt to the lanes in 16-byte pieces, and the pieces chosen so that the
// 8 lanes that shared memory serves at a time meet 8 different ones of the
// 128-byte swizzle; neighbouring keys of V are paired by byte permutes.
//
// Each warp keeps its own running max and sum (with more than 16 rows, two
// warps share the keys, one for each 16 rows).  The partial results of the
// warps and of the prefix's splits meet at the end:
//   m* = max m_s, l* = sum l_s 2^(m_s - m*), O = sum O_s 2^(m_s - m*) / l*.
// With few sequences and many own keys these are split over several blocks,
// and fa_paged_merge_kernel joins them instead.
#pragma once

#include "fa_paged.cuh"

namespace fa {

constexpr uint32_t kKernPrefixOwn = 14;
constexpr int kOwnWarps = 4;
constexpr int kOwnThreads = 32 * kOwnWarps;

constexpr int kOwnStages = 2;
constexpr int kOwnStageBytes = 8192;  // K, then V: two boxes of 16 rows x 128 bytes each

struct OwnParams {
  PagedParams p;        // the prefix pass: sizes, its partial results, o, lse
  CUtensorMap tm_k;     // [num_pages * Hkv][P][d], box 64 x 16
  CUtensorMap tm_v;
  const void* q;        // [B][Hq][N][d]
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

// Shared memory (from a 1024-byte boundary): the warps' rings, whose memory
// takes their O [16][d] at the end; (m, l) of the warps' rows; the joined
// rows' 1 / l, weights of the warps' and the prefix splits' results; barriers.
constexpr int kOwnRing = kOwnWarps * kOwnStages * kOwnStageBytes;
constexpr int kOwnFixed = kOwnRing + kOwnWarps * 16 * 8 + 32 * 4 + 32 * kOwnWarps * 4 + kOwnWarps * kOwnStages * 8;
inline int own_smem(int rows, int slots) { return 1024 + kOwnFixed + rows * slots * 4; }

// WM: warps that share a group of keys, one for each 16 rows.
template <int HD, bool BF16, int WM>
__global__ void __launch_bounds__(kOwnThreads, 3) fa_prefix_own_kernel(const __grid_constant__ OwnParams a) {
  using T = typename std::conditional<BF16, __nv_bfloat16, __half>::type;
  const PagedParams& p = a.p;
  constexpr int kC = HD / 32;         // 16-byte pieces of a lane's K (or Q) row
  constexpr int kH = HD / 64;         // 128-byte pieces of a row
  constexpr int kSub = 128 / HD;      // groups of 16 keys in a stage
  constexpr int kW = kOwnWarps / WM;  // warps along the keys
  extern __shared__ uint8_t own_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(own_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  float2* sML = reinterpret_cast<float2*>(sm + kOwnRing);
  float* sInv = reinterpret_cast<float*>(sML + kOwnWarps * 16);
  float* sWarpW = sInv + 32;                   // [row][warp along the keys]
  uint64_t* bars = reinterpret_cast<uint64_t*>(sWarpW + 32 * kOwnWarps);
  float* sW = reinterpret_cast<float*>(bars + kOwnWarps * kOwnStages);  // [row][slot]
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int nn = lane >> 2, qd = lane & 3;
  const int kw = warp / WM, mt = warp % WM;
  const int split = blockIdx.x % a.S, item = blockIdx.x / a.S;
  const int b = item / p.Hkv, g = item % p.Hkv;
  const int R = p.G * p.N;
  uint8_t* ring = sm + warp * kOwnStages * kOwnStageBytes;
  uint64_t* full = bars + warp * kOwnStages;
  if (lane == 0) {
    for (int s = 0; s < kOwnStages; ++s) mbar_init(&full[s], 1);
    fence_mbar_init();
  }
  __syncwarp();

  // The inputs were written before the prefix kernel started (it waits for
  // them before it lets this kernel be scheduled); only its results are
  // waited for, at the end.
  if (!a.follows) grid_dependency_wait();
  grid_launch_dependents();

  const int L = p.lens[b];
  const bool bad = L != 0 && (L < p.N || L > static_cast<long long>(p.max_pages) * p.P);
  if (bad && g == 0 && split == 0 && threadIdx.x == 0) record_error(kStatusBadInput, kKernPrefixOwn, 0, 0);
  // stages of 16 kSub keys: of the sequence's own part, of this split, of this warp
  constexpr int kKeys = 16 * kSub;
  const int own = bad || L <= p.prefix ? 0 : L - p.prefix;
  const int n_all = (own + kKeys - 1) / kKeys;
  const int g0 = static_cast<int>(static_cast<long long>(n_all) * split / a.S);
  const int g1 = static_cast<int>(static_cast<long long>(n_all) * (split + 1) / a.S);
  const int n_mine = g1 - g0 > kw ? (g1 - g0 - kw + kW - 1) / kW : 0;
  auto first_key = [&](int i) { return p.prefix + kKeys * (g0 + kw + i * kW); };
  // Table entries of 16 / P-th keys: lane x holds that of group x of the
  // warp's next 32 groups of 16 keys.
  const int* row = p.table + static_cast<size_t>(b) * p.max_pages;
  auto entry = [&](int grp) {
    const int key = first_key(grp / kSub) + 16 * (grp % kSub);
    return grp < n_mine * kSub && key < L ? __ldg(row + key / p.P) : -1;
  };
  int cur = entry(lane);
  auto issue = [&](int i) {
    if (i > 0 && i * kSub % 32 == 0) cur = entry(i * kSub + lane);
    uint8_t* dst = ring + (i % kOwnStages) * kOwnStageBytes;
    uint64_t* bar = &full[i % kOwnStages];
    if (lane == 0) mbar_expect_tx(bar, kOwnStageBytes);
    __syncwarp();
#pragma unroll
    for (int sub = 0; sub < kSub; ++sub) {
      const int key = first_key(i) + 16 * sub;
      const int phys = __shfl_sync(0xffffffffu, cur, (i * kSub + sub) & 31);
      int outer = -1;  // outside the tensor: zeros
      if (key < L) {
        if (phys >= 0 && phys < p.num_pages)
          outer = phys * p.Hkv + g;
        else if (lane == 0)
          record_error(kStatusBadInput, kKernPrefixOwn, 0, 1);
      }
      if (lane < 2 * kH) {  // lanes: K or V, chunk
        const int c = lane % kH, is_v = lane / kH;
        tma_load_3d(dst + is_v * (kOwnStageBytes / 2) + (kH == 2 ? c : sub) * 2048, is_v ? &a.tm_v : &a.tm_k, bar, c * 64,
                    key % p.P, outer);
      }
    }
  };
  for (int i = 0; i < kOwnStages && i < n_mine; ++i) issue(i);

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
      if (r < R) w = *reinterpret_cast<const uint4*>(q + static_cast<size_t>(r) * HD + (c >> 1) * 64 + (2 * qd + (c & 1)) * 8);
      qa[c][0][e] = w.x, qa[c][0][e + 2] = w.y, qa[c][1][e] = w.z, qa[c][1][e + 2] = w.w;
    }
  }

  float o[8 * kH][4];
#pragma unroll
  for (int j = 0; j < 8 * kH; ++j)
#pragma unroll
    for (int e = 0; e < 4; ++e) o[j][e] = 0.f;
  float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};

  bool ok = true;
  for (int i = 0; ok && i < n_mine; ++i) {
    const int st = i % kOwnStages;
    ok = __all_sync(0xffffffffu, mbar_wait_drain(&full[st], (i / kOwnStages) & 1, kKernPrefixOwn, warp, 2));
    if (!ok) break;
    const uint8_t* sk = ring + st * kOwnStageBytes;
    const uint8_t* sv = sk + kOwnStageBytes / 2;
#pragma unroll
    for (int sub = 0; sub < kSub; ++sub) {
    const int key_lo = first_key(i) + 16 * sub;
    if (key_lo >= L) break;
    float s[2][4];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      s[j][0] = s[j][1] = s[j][2] = s[j][3] = 0.f;
#pragma unroll
      for (int c = 0; c < kC; ++c) {
        const uint4 kf = *reinterpret_cast<const uint4*>(sk + (kH == 2 ? c >> 1 : sub) * 2048 + (8 * j + nn) * 128 +
                                                         (((2 * qd + (c & 1)) ^ nn) << 4));
        mma_16816<BF16>(s[j], qa[c][0], kf.x, kf.y);
        mma_16816<BF16>(s[j], qa[c][1], kf.z, kf.w);
      }
    }
    uint4 vf[4][kH];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int key = 2 * qd + (e & 1) + 8 * (e >> 1);
#pragma unroll
      for (int c = 0; c < kH; ++c) {
        vf[e][c] = *reinterpret_cast<const uint4*>(sv + (kH == 2 ? c : sub) * 2048 + key * 128 + ((nn ^ (key & 7)) << 4));
        // slots without a token may hold anything: their values count as zero
        if (key_lo + key >= L) vf[e][c] = make_uint4(0u, 0u, 0u, 0u);
      }
    }
    // scores in log2 units, hidden keys -inf: element 2e + x is row e
    const int key0 = key_lo + 2 * qd;
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
    }
    __syncwarp();  // every lane has read the stage
    if (i + kOwnStages < n_mine) issue(i + kOwnStages);
  }

  // The warp's rows into its ring: lane holds features c 64 + qd 16 + i
  // (element 0 of o[8 c + i]; + 8: element 1) of rows nn (and + 8: 2, 3).
  float* sO = reinterpret_cast<float*>(ring);
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    l[e] += __shfl_xor_sync(0xffffffffu, l[e], 1);
    l[e] += __shfl_xor_sync(0xffffffffu, l[e], 2);
    const int r = nn + 8 * e;
    if (qd == 0) sML[warp * 16 + r] = make_float2(m[e], l[e]);
    if (mt * 16 + r < R)
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
  const bool last = a.S == 1;
  if (last && a.follows) grid_dependency_wait();  // the prefix's partial results
  __syncthreads();
  // Weights of a row's partial results: a warp takes rows in turn, its lanes
  // the prefix's splits.
  const int tile = b / p.seqs;
  const bool single = (p.n_tiles & 1) && tile == p.n_tiles - 1;
  const int slots = last ? (single ? p.S_single : p.S) : 0;  // 0 without a prefix
  const long long part = (static_cast<long long>(g) * p.n_tiles + tile) * p.slots;
  auto tile_row = [&](int r) {  // of the prefix's tile: (sequence, token, head)
    return ((b % p.seqs) * p.N + r % p.N) * p.G + r / p.N;
  };
  const long long out0 = (static_cast<long long>(b) * p.Hkv + g) * R;
  for (int r = warp; r < R; r += kOwnWarps) {
    const float2* ml = p.part_ml + part * 128 + tile_row(r);
    float2 mine = make_float2(-INFINITY, 0.f);
    if (lane < kW) mine = sML[(lane * WM + r / 16) * 16 + r % 16];
    float ms = mine.x;
    for (int s = lane; s < slots; s += 32) ms = fmaxf(ms, ml[s * 128].x);
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) ms = fmaxf(ms, __shfl_xor_sync(0xffffffffu, ms, x));
    const float ref = ms == -INFINITY ? 0.f : ms;
    float w = ex2_approx(mine.x - ref);
    if (lane < kW) sWarpW[r * kOwnWarps + lane] = w;
    float ls = mine.y * w;
    for (int s = lane; s < slots; s += 32) {
      const float2 y = ml[s * 128];
      w = ex2_approx(y.x - ref);
      sW[r * slots + s] = w;
      ls += y.y * w;
    }
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) ls += __shfl_xor_sync(0xffffffffu, ls, x);
    if (lane == 0) {
      sInv[r] = !last ? 1.f : ls > 0.f ? 1.f / ls : 0.f;
      if (last)
        p.lse[out0 + r] = ls > 0.f ? (ms + __log2f(ls)) * 0.69314718055994531f : -INFINITY;
      else
        reinterpret_cast<float2*>(a.own_ml)[(out0 + r) * a.S + split] = make_float2(ms, ls);
    }
  }
  __syncthreads();
  for (int x = threadIdx.x; x < R * (HD / 4); x += kOwnThreads) {
    const int r = x / (HD / 4), c4 = x % (HD / 4);
    const float4* po = p.part_o + (part * (HD / 4) + c4) * 128 + tile_row(r);
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    auto add = [&](float w, const float4* src) {
      if (w == 0.f) return;  // nothing there (an empty split leaves its O unwritten)
      const float4 z = *src;
      acc.x += z.x * w, acc.y += z.y * w, acc.z += z.z * w, acc.w += z.w * w;
    };
#pragma unroll 8
    for (int s = 0; s < slots; ++s) add(sW[r * slots + s], po + static_cast<long long>(s) * (HD / 4) * 128);
#pragma unroll
    for (int w = 0; w < kW; ++w)
      add(sWarpW[r * kOwnWarps + w],
          reinterpret_cast<const float4*>(sm + (w * WM + r / 16) * kOwnStages * kOwnStageBytes) + (r % 16) * (HD / 4) + c4);
    const float inv = sInv[r];
    acc.x *= inv, acc.y *= inv, acc.z *= inv, acc.w *= inv;
    if (last) {
      uint2 w;
      w.x = pack2<BF16>(acc.x, acc.y);
      w.y = pack2<BF16>(acc.z, acc.w);
      *reinterpret_cast<uint2*>(static_cast<T*>(p.o) + (out0 + r) * HD + 4 * c4) = w;
    } else {
      reinterpret_cast<float4*>(a.own_o + ((out0 + r) * a.S + split) * HD)[c4] = acc;
    }
  }
  // the prefix kernel, too, is complete before this one is: whoever waits for
  // this kernel may read what both left
  if (a.S > 1 && a.follows) grid_dependency_wait();
}

}  // namespace fa
