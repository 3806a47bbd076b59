// The second half of decode behind a shared prefix: every sequence's own keys
// (those behind the prefix), joined with the prefix's partial results that
// fa_paged_kernel left in the workspace.
//
// A block takes the R = G Nq <= 32 rows of one (sequence, kv head).  Each
// cached byte is used once, for R rows, so the work is bound by memory and,
// sequences' own parts being short, by latency.  A warp therefore runs its
// own ring of stages (K and V rows of 16 keys; as many stages as the blocks on
// an SM leave room for), with no barrier between warps until the end, and
// 16 x 16 fragments go from shared memory to mma.sync: 16 rows are one of its
// tiles, and a stage 32 of its instructions at d = 128.  The stages are filled
// by 16-byte asynchronous copies of all lanes (as TMA boxes of 16 rows x 128
// bytes, four a stage, they measured the same, near what an SM's TMA engine
// takes: some 40 ns a box).  (tcgen05 takes 128 rows or keys at a time and its
// result through tensor memory: the decode kernel built on it needs about 4 us
// for a sequence of 150 keys however few its rows are.)
// A warp's time is its instructions (two or three warps share a scheduler), so
// a stage is kept to about 150 of them: fragments by ldmatrix from 128-byte
// swizzled rows, a reference max that moves only when a score exceeds it by
// more than 8 (log2), the mask, the clearing of rows without a token and the
// table look-up outside the common path.
//
// Probabilities are rounded to the I/O type for mma.sync, as in the row-tile
// kernel, and bounded by 2^8; l, O and what is joined are in 32 bits.
//
// Each warp keeps its own running max and sum (with more than 16 rows, two
// warps share the keys, one for each 16 rows).  The partial results of the
// warps and of the prefix's splits meet at the end:
//   m* = max m_s, l* = sum l_s 2^(m_s - m*), O = sum O_s 2^(m_s - m*) / l*.
// With few sequences and many own keys these are split over several blocks,
// and fa_paged_merge_kernel joins them instead.  A short prefix is taken with
// the own keys, by every sequence again (from L2): one kernel instead of two.
//
// 96 sequences x 8 heads of 500 own keys on average (196 MB): 40-42 us behind
// the prefix pass, 4.8 TB/s; 50 x 12 of 150 keys of 64: 13.4 us, most of it
// the first loads behind the prefix kernel's end and the join (3 us).
#pragma once

#include "fa_paged.cuh"

namespace fa {

constexpr uint32_t kKernPrefixOwn = 14;
constexpr int kOwnWarps = 4;
constexpr int kOwnThreads = 32 * kOwnWarps;

constexpr int kOwnMaxStages = 8;
// a stage: K, then V rows of 16 keys
__host__ __device__ constexpr int own_stage_bytes(int d) { return 2 * 16 * d * 2; }
// blocks that an SM's registers hold
__host__ __device__ constexpr int own_blocks_per_sm(int d) { return d == 128 ? 3 : 4; }

struct OwnParams {
  PagedParams p;        // the prefix pass: sizes, its partial results, o, lse
  const void* q;        // [B][Hq][N][d]
  const void* k_cache;  // [num_pages][Hkv][P][d]
  const void* v_cache;
  float* own_o;         // [row][S][d], [row][S][2]: with S > 1
  float* own_ml;
  int S;
  int stages;           // of a warp's ring
  int log2P;            // log2 of the page size
  int shared_pages;     // pages found through sequence 0's table (a short prefix, taken with the own keys)
};

// 16 bytes global -> shared, the bytes behind the first `bytes` as zeros.
__device__ __forceinline__ void copy16_async(uint32_t dst, const void* src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
// Arrives on `bar` once this thread's copies so far have landed.
__device__ __forceinline__ void copies_arrive(uint64_t* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}

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
// rows' 1 / l, weights of the warps' results; barriers; weights of the prefix
// splits' results.
constexpr int kOwnFixed = kOwnWarps * 16 * 8 + 32 * 4 + 32 * kOwnWarps * 4 + kOwnWarps * kOwnMaxStages * 8;
inline int own_smem(int d, int stages, int rows, int slots) {
  return 1024 + kOwnWarps * stages * own_stage_bytes(d) + kOwnFixed + rows * slots * 4;
}

constexpr int kOwnSmemLimit = 227 * 1024;

__device__ __forceinline__ void ldmatrix_x4(uint32_t* r, uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldmatrix_x4_trans(uint32_t* r, uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}

// WM: warps that share a group of keys, one for each 16 rows.
template <int HD, bool BF16, int WM>
__global__ void __launch_bounds__(kOwnThreads, own_blocks_per_sm(HD)) fa_prefix_own_kernel(const __grid_constant__ OwnParams a) {
  using T = typename std::conditional<BF16, __nv_bfloat16, __half>::type;
  const PagedParams& p = a.p;
  constexpr int kStage = own_stage_bytes(HD);
  constexpr int kSteps = HD / 16;     // inner steps of a score
  constexpr int kW = kOwnWarps / WM;  // warps along the keys
  constexpr float kSlack = 8.f;
  extern __shared__ uint8_t own_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(own_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const int NS = a.stages;
  float2* sML = reinterpret_cast<float2*>(sm + kOwnWarps * NS * kStage);
  float* sInv = reinterpret_cast<float*>(sML + kOwnWarps * 16);
  float* sWarpW = sInv + 32;                   // [row][warp along the keys]
  uint64_t* bars = reinterpret_cast<uint64_t*>(sWarpW + 32 * kOwnWarps);
  float* sW = reinterpret_cast<float*>(bars + kOwnWarps * kOwnMaxStages);  // [row][slot]
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int nn = lane >> 2, qd = lane & 3;
  const int kw = warp / WM, mt = warp % WM;
  const int split = blockIdx.x % a.S, item = blockIdx.x / a.S;
  const int b = item / p.Hkv, g = item % p.Hkv;
  const int R = p.G * p.N;
  const uint32_t ring = smem_u32(sm) + warp * NS * kStage;
  uint64_t* full = bars + warp * kOwnMaxStages;
  if (lane == 0) {
    for (int s = 0; s < NS; ++s) mbar_init(&full[s], 32);
    fence_mbar_init();
  }
  __syncwarp();

  // Before anything is read, the inputs included: those of a step come from the
  // append in front of the prefix kernel, and that an earlier kernel's writes
  // are visible is promised only to a kernel that has waited.
  grid_dependency_wait();
  grid_launch_dependents();

  const int L = p.lens[b];
  const bool bad = L != 0 && (L < p.N || L > static_cast<long long>(p.max_pages) * p.P);
  if (bad && g == 0 && split == 0 && threadIdx.x == 0) record_error(kStatusBadInput, kKernPrefixOwn, 0, 0);
  // groups of 16 keys: of the sequence's own part, of this split, of this warp
  const int own = bad || L <= p.prefix ? 0 : L - p.prefix;
  const int n_all = (own + 15) / 16;
  const int g0 = a.S == 1 ? 0 : static_cast<int>(static_cast<long long>(n_all) * split / a.S);
  const int g1 = a.S == 1 ? n_all : static_cast<int>(static_cast<long long>(n_all) * (split + 1) / a.S);
  const int n_mine = g1 - g0 > kw ? (g1 - g0 - kw + kW - 1) / kW : 0;
  auto first_key = [&](int i) { return p.prefix + 16 * (g0 + kw + i * kW); };
  // Table entries of the warp's groups, 32 at a time, one a lane (unsplit, the
  // first ones are asked for before the length is known; by plain loads, as in
  // the row-tile kernel).
  const int* row = p.table + static_cast<size_t>(b) * p.max_pages;
  auto entry = [&](int i) {
    // (unsigned: a group behind the last one may pass 2^31)
    const uint32_t page = (static_cast<uint32_t>(p.prefix) + 16u * static_cast<uint32_t>(g0 + kw + i * kW)) >> a.log2P;
    const int* from = page < static_cast<uint32_t>(a.shared_pages) ? p.table : row;
    return page < static_cast<uint32_t>(p.max_pages) ? from[page] : -1;
  };
  int cur = entry(lane);

  // A stage: 16 rows of K, then of V, contiguous in the cache; in shared
  // memory chunks of 64 features [16][128 bytes], 16-byte pieces swizzled by
  // row.  Lane: 16 bytes of every 512.
  constexpr int kRowLanes = HD / 8, kRows = 32 / kRowLanes;  // lanes of a row, rows of a copy
  const int lr = lane / kRowLanes;
  uint32_t to[8 / kRows];  // where the lane's piece goes, for rows lr, lr + kRows, .. below 8
#pragma unroll
  for (int x = 0; x < 8 / kRows; ++x) {
    const int piece = lane % kRowLanes, r = x * kRows + lr;
    to[x] = (piece >> 3) * 2048 + r * 128 + (((piece & 7) ^ r) << 4);
  }
  const T* kc = static_cast<const T*>(a.k_cache) + lane * 8;
  const T* vc = static_cast<const T*>(a.v_cache) + lane * 8;
  const uint32_t ring_end = ring + NS * kStage;
  uint32_t dst = ring;  // stage of the next group to load
  uint64_t* dst_bar = full;
  auto issue = [&](int i) {
    if (i > 0 && i % 32 == 0) cur = entry(i + lane);
    const int key = first_key(i);
    const int phys = __shfl_sync(0xffffffffu, cur, i & 31);
    const bool page_ok = phys >= 0 && phys < p.num_pages;
    if (page_ok && key + 16 <= L) {
      const long long src = ((static_cast<long long>(phys) * p.Hkv + g) * p.P + (key & (p.P - 1))) * HD;
#pragma unroll
      for (int x = 0; x < 16 / kRows; ++x) {
        const uint32_t t = dst + to[x % (8 / kRows)] + x / (8 / kRows) * 1024;
        copy16_async(t, kc + src + x * 256, 16);
        copy16_async(t + kStage / 2, vc + src + x * 256, 16);
      }
    } else {
      // rows without a token, which may hold anything, become zeros
      if (!page_ok && lane == 0) record_error(kStatusBadInput, kKernPrefixOwn, 0, 1);
      const long long src = page_ok ? ((static_cast<long long>(phys) * p.Hkv + g) * p.P + (key & (p.P - 1))) * HD : 0;
#pragma unroll 1
      for (int x = 0; x < 16 / kRows; ++x) {
        const int r = x * kRows + lr, piece = lane % kRowLanes;
        const uint32_t t = dst + (piece >> 3) * 2048 + r * 128 + (((piece & 7) ^ (r & 7)) << 4);
        const int bytes = page_ok && key + r < L ? 16 : 0;
        copy16_async(t, kc + src + x * 256, bytes);
        copy16_async(t + kStage / 2, vc + src + x * 256, bytes);
      }
    }
    copies_arrive(dst_bar);
    dst += kStage, ++dst_bar;
    if (dst == ring_end) dst = ring, dst_bar = full;
  };
  for (int i = 0; i < NS && i < n_mine; ++i) issue(i);

  // Q: rows mt * 16 + nn and + 8 as the A operand
  const T* q = static_cast<const T*>(a.q) + (static_cast<size_t>(b) * p.Hkv + g) * R * HD;
  uint32_t qa[kSteps][4];
  int lim[2];  // last key the two rows see
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const int r = mt * 16 + nn + 8 * e;
    lim[e] = L - p.N + r % p.N;
#pragma unroll
    for (int k = 0; k < kSteps; ++k) {
      qa[k][e] = qa[k][e + 2] = 0u;
      if (r < R) {
        const uint32_t* src = reinterpret_cast<const uint32_t*>(q + static_cast<size_t>(r) * HD + k * 16 + 2 * qd);
        qa[k][e] = src[0];
        qa[k][e + 2] = src[4];
      }
    }
  }

  float o[HD / 8][4];  // features 8 j + 2 qd, + 1 of rows nn (0, 1) and nn + 8 (2, 3)
#pragma unroll
  for (int j = 0; j < HD / 8; ++j)
#pragma unroll
    for (int e = 0; e < 4; ++e) o[j][e] = 0.f;
  float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
  const float c_log2 = p.scale_log2;

  // the lane's row addresses for ldmatrix: K keys l & 7 (+ 8: lanes 16 up),
  // pieces 0, 1; V keys l & 15, pieces 0, 1
  const int k_key = (lane & 7) + 8 * (lane >> 4), v_key = lane & 15;
  const uint32_t k_off = k_key * 128 + ((((lane >> 3) & 1) ^ (k_key & 7)) << 4);
  const uint32_t v_off = v_key * 128 + (((lane >> 4) ^ (v_key & 7)) << 4) + kStage / 2;

  uint32_t st = ring;  // stage of group i
  uint64_t* st_bar = full;
  uint32_t phase = 0;
  for (int i = 0; i < n_mine; ++i) {
    if (!__all_sync(0xffffffffu, mbar_wait_drain(st_bar, phase, kKernPrefixOwn, warp, 2))) break;
    float s[2][4], s2[2][4];  // two sums: four chains of MMAs side by side
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) s[j][e] = s2[j][e] = 0.f;
#pragma unroll
    for (int k = 0; k < kSteps; ++k) {
      uint32_t kf[4];
      ldmatrix_x4(kf, (st + k_off + (k >> 2) * 2048) ^ ((k & 3) << 5));
      mma_16816<BF16>(k & 1 ? s2[0] : s[0], qa[k], kf[0], kf[1]);
      mma_16816<BF16>(k & 1 ? s2[1] : s[1], qa[k], kf[2], kf[3]);
    }
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) s[j][e] += s2[j][e];
    const int key_lo = first_key(i);
    if (key_lo + 15 > L - p.N) {  // keys that some row does not see
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (key_lo + 8 * j + 2 * qd + (e & 1) > lim[e >> 1]) s[j][e] = -INFINITY;
    }
    float mx[2];
#pragma unroll
    for (int e = 0; e < 2; ++e)
      mx[e] = fmaxf(fmaxf(s[0][2 * e], s[0][2 * e + 1]), fmaxf(s[1][2 * e], s[1][2 * e + 1])) * c_log2;
    if (__any_sync(0xffffffffu, mx[0] > m[0] + kSlack || mx[1] > m[1] + kSlack)) {
      float fac[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        mx[e] = fmaxf(mx[e], __shfl_xor_sync(0xffffffffu, mx[e], 1));
        mx[e] = fmaxf(mx[e], __shfl_xor_sync(0xffffffffu, mx[e], 2));
        mx[e] = fmaxf(mx[e], m[e]);
        fac[e] = mx[e] == -INFINITY ? 1.f : ex2_approx(m[e] - mx[e]);
        l[e] *= fac[e];
        m[e] = mx[e];
      }
#pragma unroll
      for (int j = 0; j < HD / 8; ++j) {
        o[j][0] *= fac[0], o[j][1] *= fac[0];
        o[j][2] *= fac[1], o[j][3] *= fac[1];
      }
    }
    const float ref[2] = {m[0] == -INFINITY ? 0.f : m[0], m[1] == -INFINITY ? 0.f : m[1]};
    uint32_t pa[4];
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float x = ex2_approx(fmaf(s[j][2 * e], c_log2, -ref[e])), y = ex2_approx(fmaf(s[j][2 * e + 1], c_log2, -ref[e]));
        l[e] += x + y;
        pa[2 * j + e] = pack2<BF16>(x, y);
      }
#pragma unroll
    for (int j = 0; j < HD / 8; j += 2) {
      uint32_t vf[4];
      ldmatrix_x4_trans(vf, (st + v_off + (j >> 3) * 2048) ^ ((j & 7) << 4));
      mma_16816<BF16>(o[j], pa, vf[0], vf[1]);
      mma_16816<BF16>(o[j + 1], pa, vf[2], vf[3]);
    }
    __syncwarp();  // every lane has read the stage
    if (i + NS < n_mine) issue(i + NS);
    st += kStage, ++st_bar;
    if (st == ring_end) st = ring, st_bar = full, phase ^= 1;
  }
  // nothing is in flight here, unless a wait above ran out
  asm volatile("cp.async.wait_all;" ::: "memory");
  __syncwarp();

  // The warp's rows into its ring.
  float* sO = reinterpret_cast<float*>(sm + warp * NS * kStage);
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    l[e] += __shfl_xor_sync(0xffffffffu, l[e], 1);
    l[e] += __shfl_xor_sync(0xffffffffu, l[e], 2);
    const int r = nn + 8 * e;
    if (qd == 0) sML[warp * 16 + r] = make_float2(m[e], l[e]);
    if (mt * 16 + r < R)
#pragma unroll
      for (int j = 0; j < HD / 8; ++j)
        *reinterpret_cast<float2*>(sO + r * HD + 8 * j + 2 * qd) = make_float2(o[j][2 * e], o[j][2 * e + 1]);
  }
  const bool last = a.S == 1;
  __syncthreads();
  // Weights of a row's partial results: a warp takes rows in turn, its lanes
  // the prefix's splits.
  const int tile = b / p.seqs;
  const bool single = tile >= 2 * p.n_pairs;
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
      sInv[r] = !last ? 1.f : ls != 0.f ? 1.f / ls : 0.f;  // (NaN shows)
      if (last)
        p.lse[out0 + r] = ls != 0.f ? (ms + __log2f(ls)) * 0.69314718055994531f : -INFINITY;
      else
        reinterpret_cast<float2*>(a.own_ml)[(out0 + r) * a.S + split] = make_float2(ms, ls);
    }
  }
  __syncthreads();
  for (int x = threadIdx.x; x < R * (HD / 4); x += kOwnThreads) {
    const int r = x % R, c4 = x / R;  // rows fastest: neighbours in the prefix's partial results
    const float4* po = p.part_o + (part * (HD / 4) + c4) * 128 + tile_row(r);
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    auto add = [&](float w, const float4* src) {
      const float4 z = *src;
      acc.x += z.x * w, acc.y += z.y * w, acc.z += z.z * w, acc.w += z.w * w;
    };
#pragma unroll 8
    for (int s = 0; s < slots; ++s) add(sW[r * slots + s], po + static_cast<long long>(s) * (HD / 4) * 128);
#pragma unroll
    for (int w = 0; w < kW; ++w)
      add(sWarpW[r * kOwnWarps + w],
          reinterpret_cast<const float4*>(sm + (w * WM + r / 16) * NS * kStage) + (r % 16) * (HD / 4) + c4);
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
}

}  // namespace fa
