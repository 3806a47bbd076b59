// Attention of many query rows over a paged key/value cache: the forward pass
// of new tokens (fa_fwd_paged) and the prefix part of a decode step whose
// sequences share their first pages (fa_decode_prefix).  Both are the forward
// pass's product chain (S = Q K^T, online softmax, O += P V; all in tensor
// memory) over keys found through a block table; they differ in which rows
// make up a tile.
//
// A row tile is 128 rows of one kv head that see the same keys:
//   forward   toks = 128 / G consecutive new tokens of one sequence times the
//             G = Hq / Hkv query heads of the group, token-major, so that a
//             tile's rows end at nearly the same key and the group's heads
//             share each key read;
//   prefix    seqs = 128 / (G N) sequences times their G N rows: the whole
//             batch reads each prefix key once per row tile, or once per two
//             where they are taken in pairs.
// Either is one box of a 5-D tensor map over q (feature, head of the group,
// token, kv head, sequence).
//
// A thread block takes two row tiles of a kv head (a pair) or one (the last of
// an odd number, and each while there are too few to fill the GPU), and a
// range of 128-key tiles:
//   pair      row tile t belongs to softmax warpgroup t, both read every key
//             tile: step i is row tile i & 1 on key tile i >> 1;
//   single    both warpgroups hold the same rows and take turns on the key
//             tiles: step i is warpgroup i & 1 on key tile i; their two
//             partial results are joined in shared memory at the end.
// The tensor cores run the scores two or three steps ahead: one warpgroup's
// softmax overlaps the other's products in both forms.
//
// When there are too few blocks to fill the GPU the key tiles of a row tile are
// split over several blocks, each leaving unnormalised O with its reference
// max m and sum l (base 2) in the workspace; fa_paged_merge_kernel joins them
// (and the partial results of each sequence's own keys):
//   m* = max m_s, l* = sum l_s 2^(m_s - m*), O = sum O_s 2^(m_s - m*) / l*.
//
// Warp roles (384 threads) and the register split are those of the forward
// kernel: softmax warpgroups 0 and 1, MMA warp 8, TMA warps 9 (K) and 10 (V).
// A key tile is 128 / P page boxes; a TMA warp holds 32 table entries in its
// lanes, and the lanes of a tile's pages issue its copies side by side.
//
// Slots behind a sequence's last token may hold anything, NaN included: scores
// of hidden keys are replaced, and the value rows of such slots are cleared
// in shared memory before the product reads them (0 * NaN is not 0).
//
// The probabilities are rounded to the I/O type for the P V product: the tensor
// core takes 16-bit operands (tf32 would halve its rate and double P's room in
// tensor memory).  The sums l are of the unrounded values, O stays in 32 bits
// until it is written.  Against 64 bits O is off by 2.3e-3 relative in bf16 and
// 2.9e-4 in fp16; rounding O alone costs 1.7e-3 and 2.1e-4.
//
// What bounds it: with many row tiles the chain softmax -> P V -> next S of a
// row tile, 1.1 + 0.9 us, two tiles in flight: 1.04 us a step at d = 128 (two
// prompts of 4096 tokens behind 6299 and 7983 cached ones, 32 heads: 1055-1075
// us, 1150-1170 TFLOP/s, in short runs; 1240 us, 995 TFLOP/s, at the clock of a
// long one); with one, memory and the block's start and end (16 384 shared keys
// of 8 heads, 67 MB, in 19-22 us).  The TMA engine takes about 40 ns a box: K and
// V tiles are issued by a warp each, started before the block's other warps are
// set up.  168 registers a thread at launch, 36 bytes of spills.
#pragma once

#include <type_traits>

#include "fa_decode.cuh"  // programmatic dependent launch, kStatusBadInput
#include "fa_fwd.cuh"     // FwdLayout, register split, kRefSlack

namespace fa {

constexpr uint32_t kKernPaged = 13;
constexpr int kPagedTile = 128;  // rows of a row tile, keys of a key tile

struct PagedParams {
  CUtensorMap tm_q;  // q as (d, G, N, Hkv, B), box 64 x G x toks x 1 x seqs
  CUtensorMap tm_k;  // [num_pages * Hkv][P][d], box 64 x P
  CUtensorMap tm_v;
  const int* table;     // [B][max_pages]
  const int* lens;      // [B]
  const int* new_lens;  // [B] or nullptr: N each
  void* o;              // [B][Hq][N][d], written here when part_o is nullptr
  float* lse;           // [B][Hq][N]
  float4* part_o;       // [owner][row tile][slots][d / 4][128]
  float2* part_ml;      // [owner][row tile][slots][128]: (m, l) in base 2
  int B, Hq, Hkv, G, N, P, max_pages, num_pages;
  int decode;           // 1: decode behind a prefix (a tile's rows come from several sequences); 0: forward pass
  int prefix;           // keys of the shared prefix
  int toks, seqs;       // a row tile: tokens x sequences (x G heads)
  int n_tiles;          // row tiles of an owner (kv head, of a sequence in the forward pass)
  int n_pairs;          // the first 2 n_pairs of them in pairs, the others as singles
  int S, S_single;      // key splits of a pair / of a single
  int slots;            // the larger of those in use
  float scale_log2;
};

// What a sequence's lengths allow.
struct PagedSeq {
  int L, n;     // cached tokens, new tokens
  int row_end;  // new-token rows that are written
  bool bad, live;
};

__device__ __forceinline__ PagedSeq paged_seq(const PagedParams& p, int b) {
  PagedSeq q;
  q.L = p.lens[b];
  q.n = p.new_lens ? p.new_lens[b] : p.N;
  const bool n_ok = q.n >= 0 && q.n <= p.N;
  q.bad = !n_ok || (q.L != 0 && (q.L < q.n || q.L > static_cast<long long>(p.max_pages) * p.P));
  q.live = !q.bad && q.L > 0;
  q.row_end = q.bad ? p.N : q.n;
  return q;
}

// Row r of a row tile: sequence, token and output row ((b Hq + h) N + token).
struct PagedRow {
  int b, t;
  bool in_tile;
  long long out;
};

__device__ __forceinline__ PagedRow paged_row(const PagedParams& p, int owner, int tile, int r) {
  PagedRow w;
  const int hg = r % p.G, x = r / p.G;
  if (p.decode) {
    w.b = tile * p.seqs + x / p.N;
    w.t = x % p.N;
    w.in_tile = r < p.seqs * p.N * p.G && w.b < p.B;
  } else {
    w.b = owner / p.Hkv;
    w.t = tile * p.toks + x;
    w.in_tile = r < p.toks * p.G && w.t < p.N;
  }
  w.out = (static_cast<long long>(w.b) * p.Hq + (owner % p.Hkv) * p.G + hg) * p.N + w.t;
  return w;
}

// A block's work: a pair of row tiles or a single, and a range of key tiles.
struct PagedItem {
  bool single;  // one row tile, its key tiles shared out between the warpgroups
  bool dead;    // only padding rows: nothing is written
  int split, splits, owner, tile0, g, b;
  int valid_end;  // keys that hold a token
  int k0, n_kv;   // key tiles
};

// Blocks in order: pairs first, the last tokens (most keys) of every sequence
// first; then the singles, which take half a pair's time.
__device__ __forceinline__ PagedItem paged_item(const PagedParams& p) {
  PagedItem it;
  int x = blockIdx.x;
  const int owners = p.decode ? p.Hkv : p.B * p.Hkv;
  it.single = x >= p.n_pairs * owners * p.S;
  if (it.single) x -= p.n_pairs * owners * p.S;
  it.splits = it.single ? p.S_single : p.S;
  it.split = x % it.splits;
  it.owner = (x / it.splits) % owners;
  it.tile0 = it.single ? p.n_tiles - 1 - x / (it.splits * owners) : 2 * (p.n_pairs - 1 - x / (it.splits * owners));
  it.g = it.owner % p.Hkv;
  it.b = p.decode ? 0 : it.owner / p.Hkv;
  return it;
}

// What of it depends on the sequence's lengths.
__device__ __forceinline__ void paged_item_keys(const PagedParams& p, PagedItem& it) {
  it.dead = false;
  int keys;  // keys some row of the item sees
  if (p.decode) {
    keys = it.valid_end = p.prefix;
  } else {
    const PagedSeq q = paged_seq(p, it.b);
    const int tok0 = it.tile0 * p.toks, tok1 = min(q.n, tok0 + (it.single ? 1 : 2) * p.toks);
    if (q.bad && threadIdx.x == 0 && it.split == 0 && it.g == 0) record_error(kStatusBadInput, kKernPaged, 0, 0);
    it.dead = tok0 >= q.row_end;
    keys = q.live && !it.dead ? q.L - q.n + tok1 : 0;
    it.valid_end = q.L;
  }
  const int n = (keys + kPagedTile - 1) / kPagedTile;
  it.k0 = static_cast<int>(static_cast<long long>(n) * it.split / it.splits);
  it.n_kv = static_cast<int>(static_cast<long long>(n) * (it.split + 1) / it.splits) - it.k0;
}

// Arrives on a named barrier without waiting for it.
__device__ __forceinline__ void named_barrier_arrive(uint32_t id, uint32_t count) {
  asm volatile("bar.arrive %0, %1;" ::"r"(id), "r"(count) : "memory");
}

__device__ __forceinline__ void tma_load_5d(void* dst, const CUtensorMap* map, uint64_t* bar, int32_t c0, int32_t c1,
                                            int32_t c2, int32_t c3, int32_t c4) {
  asm volatile(
      "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5, %6, %7}], [%2];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(c4)
      : "memory");
}

// Shared memory: the forward kernel's layout and, behind it, (m, l) of both
// warpgroups' rows.  Nothing is left at d = 128 to re-align the base with; the
// dynamic shared memory of a block without static shared memory starts on a
// 1024-byte boundary (checked).
template <int HD>
struct PagedLayout : FwdLayout<HD> {
  static constexpr int kOffML = (FwdLayout<HD>::kSmemBytes + 15) / 16 * 16;
  // Score buffers in tensor memory, 128 columns each, then the two O tiles: a
  // third one fits at d = 64, and lets S run three steps ahead of P V, so that
  // a warpgroup finds its next scores ready (two ahead, it waits for its own P
  // V first: 0.95 us a step, 1.1 us of softmax and 0.8 us of products in turn
  // on each of two warpgroups).
  static constexpr int kDepth = HD == 64 ? 3 : 2;
  static constexpr int kOffStep = kOffML + 2 * 128 * 8;  // s_full[kDepth], p_half[kDepth][2]
  static constexpr int kBytes = kOffStep + 3 * kDepth * 8;
  static_assert(kBytes <= 232448, "shared memory budget");
};

template <int HD, bool BF16>
__global__ void __launch_bounds__(kFwdThreads, 1) fa_paged_kernel(const __grid_constant__ PagedParams p) {
  using L = PagedLayout<HD>;
  using T = typename std::conditional<BF16, __nv_bfloat16, __half>::type;
  constexpr int NS = L::kSlots;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = smem_raw;
  uint8_t* sQ = sm + L::kOffQ;
  uint8_t* sRing = sm + L::kOffRing;
  uint64_t* bars = reinterpret_cast<uint64_t*>(sm + L::kOffBar);
  uint64_t* q_full = bars;
  uint64_t* slot_full = bars + 1;
  uint64_t* slot_empty = slot_full + NS;
  uint64_t* pv_done = slot_empty + NS;  // [warpgroup]
  uint64_t* done_bar = pv_done + 2;
  constexpr int kDepth = L::kDepth;
  constexpr uint32_t kColO = kDepth * 128;
  uint64_t* s_full = reinterpret_cast<uint64_t*>(sm + L::kOffStep);  // [buffer]
  uint64_t* p_half = s_full + kDepth;                                // [buffer][half]
  float2* sML = reinterpret_cast<float2*>(sm + L::kOffML);
  uint32_t* tmem_ptr = reinterpret_cast<uint32_t*>(sm + L::kOffTmemPtr);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(sm + L::kOffAbort);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (smem_u32(sm) & 1023u) {  // refuse
    if (tid == 0) record_error(kStatusSmemAlign, kKernPaged, 0, 0);
    return;
  }
  const int box_rows = p.G * p.toks * p.seqs;  // rows of a tile that the q box fills

  // The third warpgroup gives its registers up at once, so that the softmax
  // warpgroups need not wait for them behind the first loads.
  if (warp >= 8) setmaxnreg_dec<kFwdOtherRegs>();
  const bool produces = warp == 9 || warp == 10;
  if (produces) {
    if (warp == 9 && lane == 0) {
      mbar_init(q_full, 1);
      for (int s = 0; s < NS; ++s) {
        mbar_init(&slot_full[s], 1);
        mbar_init(&slot_empty[s], 1);
      }
      for (int i = 0; i < kDepth; ++i) {
        mbar_init(&s_full[i], 1);
        mbar_init(&p_half[2 * i], 128);
        mbar_init(&p_half[2 * i + 1], 128);
      }
      mbar_init(&pv_done[0], 1);
      mbar_init(&pv_done[1], 1);
      mbar_init(done_bar, 1);
      *abort_flag = 0;
      fence_mbar_init();
    }
    if (lane == 0) prefetch_tensormap(warp == 10 ? &p.tm_v : &p.tm_k);
    named_barrier_sync(2, 64);
    named_barrier_arrive(3, kFwdThreads);  // the others wait for the barriers, not for the first loads
  } else if (warp == 8) {
    tmem_alloc(tmem_ptr, 512);
    tmem_relinquish();
  } else {
    // rows behind the box (128 is no multiple of G toks): zeros, so that
    // their scores never move a reference
    const int i0 = warp < 8 ? tid : tid - 96;
    for (int i = i0; i < (128 - box_rows) * 8 * 2 * L::kChunks; i += 288) {
      const int box = i / ((128 - box_rows) * 8), k = i % ((128 - box_rows) * 8);
      *reinterpret_cast<uint4*>(sQ + box * L::kBoxBytes + box_rows * 128 + k * 16) = make_uint4(0u, 0u, 0u, 0u);
    }
    fence_proxy_async_smem();
  }
  grid_dependency_wait();
  grid_launch_dependents();
  uint32_t tmem = 0;
  if (!produces) {
    tc_fence_before();
    named_barrier_sync(3, kFwdThreads);
    tc_fence_after();
    tmem = *tmem_ptr;
  }

  PagedItem it = paged_item(p);
  const bool single = it.single;
  // unsplit, the first table entries are asked for before the length is known
  // (all by plain loads: the read-only path is for data that nobody writes
  // while the kernel is resident, and it is resident before its wait)
  const int* row_table = p.table + static_cast<size_t>(it.b) * p.max_pages;
  int cur = -1, nxt = -1;  // table entries of 32 pages, one a lane, and of the next 32
  if (produces && it.splits == 1) {
    if (lane < p.max_pages) cur = row_table[lane];
    if (lane + 32 < p.max_pages) nxt = row_table[lane + 32];
  }
  paged_item_keys(p, it);
  if (warp == 11) {
    // idle
  } else if (produces) {
    // ------------------------------------------------------------ producers
    // Warp 9 loads K tiles (and q), warp 10 V tiles.
    const int which = warp - 9;
    const int ppt = kPagedTile / p.P;  // pages of a key tile
    if (it.n_kv > 0) {
      const int n_pages = (it.valid_end + p.P - 1) / p.P, pg0 = it.k0 * ppt;
      auto entry = [&](int rel) { return pg0 + rel < n_pages ? row_table[pg0 + rel] : -1; };
      if (it.splits > 1) cur = entry(lane), nxt = entry(32 + lane);
      bool ok = true;
      int kt = 0;  // key tiles issued
      for (; kt < it.n_kv; ++kt) {
        const int rel = kt * ppt;
        if (kt > 0 && rel % 32 == 0) {
          cur = nxt;
          nxt = entry(rel + 32 + lane);
        }
        const int phys = __shfl_sync(0xffffffffu, cur, (rel + lane) & 31);
        int outer = -1;  // outside the tensor: the box reads as zeros
        if (lane < ppt && pg0 + rel + lane < n_pages) {
          if (phys >= 0 && phys < p.num_pages)
            outer = phys * p.Hkv + it.g;
          else
            record_error(kStatusBadInput, kKernPaged, 9, 1);
        }
        const int n = 2 * kt + which, s = n % NS;
        if (n >= NS)
          ok = __all_sync(0xffffffffu, mbar_wait(&slot_empty[s], ((n / NS) - 1) & 1, abort_flag, kKernPaged, warp, 0));
        if (!ok) break;
        if (lane == 0) mbar_expect_tx(&slot_full[s], L::kTileBytes);
        __syncwarp();
        if (lane < ppt)
          for (int c = 0; c < L::kChunks; ++c)
            tma_load_3d(sRing + s * L::kTileBytes + c * L::kBoxBytes + lane * p.P * 128, which ? &p.tm_v : &p.tm_k,
                        &slot_full[s], c * 64, 0, outer);
        if (which == 0 && kt == 0 && lane == 0) {
          const int n_q = single ? 1 : 2;
          mbar_expect_tx(q_full, static_cast<uint32_t>(n_q * L::kChunks * box_rows * 128));
          for (int t = 0; t < n_q; ++t)
            for (int c = 0; c < L::kChunks; ++c)
              tma_load_5d(sQ + t * L::kTileBytes + c * L::kBoxBytes, &p.tm_q, q_full, c * 64, 0,
                          p.decode ? 0 : (it.tile0 + t) * p.toks, it.g, p.decode ? (it.tile0 + t) * p.seqs : it.b);
        }
        __syncwarp();
      }
      // The copies in flight land before the block exits: at once, unless a
      // wait ran out (the MMA warp waits for every tile).  Then each of the
      // warp's last tiles is waited for, one whose slot the other warp filled
      // again perhaps for nothing, up to the limit of a wait.
      if (which == 0) mbar_wait_drain(q_full, 0, kKernPaged, 9, 2);
      for (int k = max(0, kt - NS); k < kt; ++k) {
        const int n = 2 * k + which;
        if (!ok || n + NS >= 2 * it.n_kv)  // else the slot was filled again: it had landed
          mbar_wait_drain(&slot_full[n % NS], (n / NS) & 1, kKernPaged, warp, 3);
      }
    }
  } else if (warp == 8) {
    // ------------------------------------------------------------ MMA issuer
    constexpr uint32_t kIdS = idesc_f16(BF16, 128, 128, false, false);
    constexpr uint32_t kIdPV = idesc_f16(BF16, 128, HD, false, true);
    const uint64_t dQ_k = sdesc_sw128(smem_u32(sQ), 16, 1024);
    const uint64_t dR_k = sdesc_sw128(smem_u32(sRing), 16, 1024);
    const uint64_t dR_mn = sdesc_sw128(smem_u32(sRing), L::kBoxBytes, 1024);
    auto wait_all = [&](uint64_t* bar, uint32_t parity, uint32_t site) -> bool {
      return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort_flag, kKernPaged, 8, site));
    };
    // ring position of step i's key tile (its value tile is the next one)
    auto ring = [&](int i) { return 2 * (single ? i : i >> 1); };
    // the last step that reads a key tile hands its slots back
    auto last_reader = [&](int i) { return single || (i & 1) != 0; };
    auto issue_s = [&](int i) -> bool {
      const int n = ring(i), s = n % NS, t = i & 1, buf = i % kDepth;
      if (!wait_all(&slot_full[s], (n / NS) & 1, 1)) return false;
      tc_fence_after();
      const uint32_t qo = single ? 0u : t * L::kTileBytes, ko = s * L::kTileBytes;
#pragma unroll
      for (int k = 0; k < HD / 16; ++k) {
        const uint32_t off = (k >> 2) * L::kBoxBytes + (k & 3) * 32;
        umma_ss_w(tmem + buf * 128, sdesc_add(dQ_k, qo + off), sdesc_add(dR_k, ko + off), kIdS, k > 0);
      }
      umma_commit_w(&s_full[buf]);
      if (last_reader(i)) umma_commit_w(&slot_empty[s]);
      return true;
    };
    auto issue_pv = [&](int i) -> bool {
      const int n = ring(i) + 1, s = n % NS, t = i & 1, j = i >> 1, buf = i % kDepth;
      if (!wait_all(&slot_full[s], (n / NS) & 1, 2)) return false;
      const uint32_t vo = s * L::kTileBytes;
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        if (!wait_all(&p_half[2 * buf + half], (i / kDepth) & 1, 3)) return false;
        tc_fence_after();
#pragma unroll
        for (int k = 4 * half; k < 4 * half + 4; ++k)
          umma_ts_w(tmem + kColO + t * HD, tmem + buf * 128 + k * 8, sdesc_add(dR_mn, vo + k * 2048), kIdPV,
                    (j > 0 || k > 0) ? 1u : 0u);
      }
      umma_commit_w(&pv_done[t]);
      if (last_reader(i)) umma_commit_w(&slot_empty[s]);
      return true;
    };
    const int steps = single ? it.n_kv : 2 * it.n_kv;
    if (steps > 0) {
      bool ok = wait_all(q_full, 0, 0);
      tc_fence_after();
      // S_0 S_1 | P_0 V, S_2 | P_1 V, S_3 | ... (two ahead; three at d = 64).
      // S overwrites the tensor memory that the O += P V before it reads P
      // from; the tensor core runs one thread's MMAs in issue order, so no wait
      // is put between them.  (One copy of each in the code: a cold instruction
      // line costs microseconds while every block's first loads are in flight.)
      for (int i = 0; ok && i < steps + kDepth; ++i) {
        if (i >= kDepth) ok = issue_pv(i - kDepth);
        if (ok && i < steps) ok = issue_s(i);
      }
    }
    // every MMA this warp issued completes before tensor memory is freed
    umma_commit_w(done_bar);
    mbar_wait_drain(done_bar, 0, kKernPaged, 8, 4);
  } else {
    setmaxnreg_inc<kFwdSoftmaxRegs>();
    // ------------------------------------------------------------ softmax
    const int t = warp >> 2;    // warpgroup
    const int r = tid & 127;    // row within the tile == tensor-memory lane
    const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
    uint32_t tm_S = tmem + t * 128 + lane_off;  // the step's score buffer
    const uint32_t tm_O = tmem + kColO + t * HD + lane_off;
    int buf = t;
    const float c_log2 = p.scale_log2;
    const uint64_t c2 = f2pack(c_log2, c_log2);
    const int tile = single ? it.tile0 : it.tile0 + t;
    const PagedRow row = paged_row(p, it.owner, tile, r);
    // last key the row sees; rows that are not written compute what they
    // find (a row never reaches another row's result)
    int lim = INT32_MAX;
    bool write = row.in_tile && !it.dead;
    if (write) {
      const PagedSeq q = paged_seq(p, row.b);
      lim = q.live ? q.L - q.n + row.t : -1;
      if (p.decode && q.live) lim = min(lim, p.prefix - 1);
      write = row.t < q.row_end;
    }
    const bool warp_works = __any_sync(0xffffffffu, write);
    const int n_mine = single ? (it.n_kv + 1 - t) / 2 : it.n_kv;
    const int n_other = it.n_kv - n_mine;  // a single's other warpgroup
    float m_ref = -INFINITY, l_sum = 0.f;
    bool ok = true;
    auto load_s = [&](int kv0, uint32_t* s) {
      tmem_ld32(tm_S + 0, s);
      tmem_ld32(tm_S + 32, s + 32);
      tmem_ld32(tm_S + 64, s + 64);
      tmem_ld32(tm_S + 96, s + 96);
      tmem_ld_wait();
      const int last = lim - kv0;  // last visible column
      if (last < 127) {
#pragma unroll
        for (int c = 0; c < 128; ++c)
          if (c > last) s[c] = __float_as_uint(-INFINITY);
      }
    };
    // P of the 32 keys 32*q4 .. +31 against the reference -m (nm2), packed to
    // 16 bits in pk[16]; the unrounded values are summed into acc.
    auto p_chunk = [&](const uint32_t* s, int q4, uint64_t nm2, uint32_t* pk, uint64_t* acc) {
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const int c = q4 * 32 + 2 * i;
        const uint64_t y = fma2(f2pack(__uint_as_float(s[c]), __uint_as_float(s[c + 1])), c2, nm2);
        const uint64_t pp = f2pack(ex2_approx(f2lo(y)), ex2_approx(f2hi(y)));
        acc[i & 3] = add2(acc[i & 3], pp);
        pk[i] = pack2<BF16>(f2lo(pp), f2hi(pp));
      }
    };
    auto hand_over = [&](int half) {
      tmem_st_wait();
      tc_fence_before();
      mbar_arrive(&p_half[2 * buf + half]);
    };
    auto sum_acc = [&](const uint64_t* acc) {
      const uint64_t a = add2(add2(acc[0], acc[1]), add2(acc[2], acc[3]));
      return f2lo(a) + f2hi(a);
    };
    for (int j = 0; j < n_mine; ++j) {
      uint32_t use = j;  // how often the buffer was used before
      if constexpr (kDepth != 2) {
        buf = (2 * j + t) % kDepth;
        use = (2 * j + t) / kDepth;
        tm_S = tmem + buf * 128 + lane_off;
      }
      if (!__all_sync(0xffffffffu, mbar_wait(&s_full[buf], use & 1, abort_flag, kKernPaged, t, 0))) {
        ok = false;
        break;
      }
      tc_fence_after();
      const int kt = single ? 2 * j + t : j;  // key tile of the block's range
      const int kv0 = (it.k0 + kt) * kPagedTile;
      if (kv0 + kPagedTile > it.valid_end && (single || t == 0)) {
        // the tile holds slots without a token: thread r clears value row r
        // if it is one (the first product on this value tile is this
        // warpgroup's, and waits for the arrivals below)
        const int n = 2 * kt + 1, s = n % NS;
        if (!__all_sync(0xffffffffu, mbar_wait(&slot_full[s], (n / NS) & 1, abort_flag, kKernPaged, t, 3))) {
          ok = false;
          break;
        }
        if (kv0 + r >= it.valid_end) {
#pragma unroll
          for (int c = 0; c < L::kChunks; ++c)
#pragma unroll
            for (int u = 0; u < 8; ++u)
              *reinterpret_cast<uint4*>(sRing + s * L::kTileBytes + c * L::kBoxBytes + r * 128 + u * 16) =
                  make_uint4(0u, 0u, 0u, 0u);
        }
        fence_proxy_async_smem();
      }
      if (!warp_works) {
        hand_over(0);
        hand_over(1);
        continue;
      }
      bool done = false;
      float m_new;
      {
        uint32_t s[128];
        load_s(kv0, s);
        // row max, eight independent chains of three-input maxima
        float mx[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) mx[i] = fmaxf(__uint_as_float(s[i]), __uint_as_float(s[8 + i]));
#pragma unroll
        for (int c = 16; c < 128; c += 16)
#pragma unroll
          for (int i = 0; i < 8; ++i)
            mx[i] = max3f(mx[i], __uint_as_float(s[c + i]), __uint_as_float(s[c + 8 + i]));
        m_new = max3f(max3f(mx[0], mx[1], mx[2]), max3f(mx[3], mx[4], mx[5]), fmaxf(mx[6], mx[7])) * c_log2;
        if (j == 0) m_ref = m_new;
        // the exponentials of keys 0-63 against the current reference do not
        // wait for the vote on the maxima (as in the forward kernel)
        const float m_use = m_ref == -INFINITY ? 0.f : m_ref;
        const uint64_t nm2 = f2pack(-m_use, -m_use);
        uint32_t pk0[16], pk1[16];
        uint64_t acc[4] = {0, 0, 0, 0};
        p_chunk(s, 0, nm2, pk0, acc);
        p_chunk(s, 1, nm2, pk1, acc);
        if (!__any_sync(0xffffffffu, m_new > m_ref + kRefSlack)) {
          tmem_st16(tm_S + 0, pk0);
          tmem_st16(tm_S + 16, pk1);
          hand_over(0);
          p_chunk(s, 2, nm2, pk0, acc);
          tmem_st16(tm_S + 32, pk0);
          p_chunk(s, 3, nm2, pk1, acc);
          tmem_st16(tm_S + 48, pk1);
          l_sum += sum_acc(acc);
          hand_over(1);
          done = true;
        }
      }
      if (done) continue;
      // A reference max must move (never in the first tile): O and l are
      // rescaled once O += P V of the previous tile is done, the tile redone.
      if (!__all_sync(0xffffffffu, mbar_wait(&pv_done[t], (j - 1) & 1, abort_flag, kKernPaged, t, 1))) {
        ok = false;
        break;
      }
      tc_fence_after();
      const float m_upd = fmaxf(m_ref, m_new);
      const float corr = m_upd == -INFINITY ? 1.f : ex2_approx(m_ref - m_upd);
      const uint64_t corr2 = f2pack(corr, corr);
      m_ref = m_upd;
      l_sum *= corr;
#pragma unroll 1
      for (int c = 0; c < HD; c += 16) {
        uint32_t o[16];
        tmem_ld16(tm_O + c, o);
        tmem_ld_wait();
#pragma unroll
        for (int i = 0; i < 16; i += 2) {
          const uint64_t v = mul2(f2pack(__uint_as_float(o[i]), __uint_as_float(o[i + 1])), corr2);
          o[i] = __float_as_uint(f2lo(v));
          o[i + 1] = __float_as_uint(f2hi(v));
        }
        tmem_st16(tm_O + c, o);
      }
      {
        uint32_t s[128];
        load_s(kv0, s);
        const float m_use = m_ref == -INFINITY ? 0.f : m_ref;
        const uint64_t nm2 = f2pack(-m_use, -m_use);
        uint64_t acc[4] = {0, 0, 0, 0};
#pragma unroll
        for (int q4 = 0; q4 < 4; ++q4) {
          uint32_t pk[16];
          p_chunk(s, q4, nm2, pk, acc);
          tmem_st16(tm_S + q4 * 16, pk);
          if (q4 == 1) hand_over(0);
        }
        l_sum += sum_acc(acc);
        hand_over(1);
      }
    }
    // ---------------------------------------------------------------- epilogue
    bool have = ok && n_mine > 0;
    if (have) have = mbar_wait(&pv_done[t], (n_mine - 1) & 1, abort_flag, kKernPaged, t, 2);
    have = __all_sync(0xffffffffu, have);
    if (!have) m_ref = -INFINITY, l_sum = 0.f;
    // A single's two partial results: tensor memory holds both in the same
    // lanes, so each warpgroup joins and writes half of the features; only
    // (m, l) go through shared memory.
    constexpr int kHalf = HD / 2;
    float w_own = 1.f, w_other = 0.f;
    bool have_other = false;
    if (single) {
      sML[t * 128 + r] = make_float2(m_ref, l_sum);
      have_other = ok && n_other > 0;
      if (have_other) have_other = mbar_wait(&pv_done[1 - t], (n_other - 1) & 1, abort_flag, kKernPaged, t, 4);
      have_other = __all_sync(0xffffffffu, have_other);
      named_barrier_sync(1, 256);
      const float2 other = sML[(1 - t) * 128 + r];
      const float m = fmaxf(m_ref, other.x);
      if (m != -INFINITY) {
        w_own = ex2_approx(m_ref - m);
        w_other = ex2_approx(other.x - m);
      }
      l_sum = l_sum * w_own + other.y * w_other;
      m_ref = m;
    }
    if (have || have_other) tc_fence_after();
    const bool seen = l_sum != 0.f;  // NaN too: scores that are no numbers show in O and lse
    const bool direct = p.part_o == nullptr;
    if (direct) {
      const float inv_l = seen ? 1.f / l_sum : 0.f;
      w_own *= inv_l;
      w_other *= inv_l;
    }
    const long long part = (static_cast<long long>(it.owner) * p.n_tiles + tile) * p.slots + it.split;
    // the rows of a tile in the I/O type, staged where q was: 16-byte pieces
    // swizzled by row (d / 8 of them; a single's half: d / 16)
    uint8_t* sOut = sQ + t * L::kTileBytes + r * (HD * 2);
    auto emit = [&](int c, const float* f) {  // features c .. c + 31 of the row
      if (direct) {
#pragma unroll
        for (int u = 0; u < 4; ++u)
          *reinterpret_cast<uint4*>(sOut + (((c / 8 + u) ^ (r & 7)) << 4)) =
              make_uint4(pack2<BF16>(f[8 * u], f[8 * u + 1]), pack2<BF16>(f[8 * u + 2], f[8 * u + 3]),
                         pack2<BF16>(f[8 * u + 4], f[8 * u + 5]), pack2<BF16>(f[8 * u + 6], f[8 * u + 7]));
      } else {
        // consecutive threads, consecutive float4: whole lines (zeros where the
        // row saw nothing: whoever joins them reads every split)
#pragma unroll
        for (int u = 0; u < 8; ++u)
          p.part_o[(part * (HD / 4) + c / 4 + u) * 128 + r] =
              make_float4(f[4 * u], f[4 * u + 1], f[4 * u + 2], f[4 * u + 3]);
      }
    };
    const int c_lo = single ? t * kHalf : 0, c_hi = single ? c_lo + kHalf : HD;
#pragma unroll 2
    for (int c = c_lo; c < c_hi; c += 32) {
      float f[32];
#pragma unroll
      for (int i = 0; i < 32; ++i) f[i] = 0.f;
      if (have) {
        uint32_t v[32];
        tmem_ld32(tm_O + c, v);
        tmem_ld_wait();
#pragma unroll
        for (int i = 0; i < 32; ++i) f[i] = __uint_as_float(v[i]) * w_own;
      }
      if (have_other) {
        uint32_t v[32];
        tmem_ld32(tmem + kColO + (1 - t) * HD + lane_off + c, v);
        tmem_ld_wait();
#pragma unroll
        for (int i = 0; i < 32; ++i) f[i] = fmaf(__uint_as_float(v[i]), w_other, f[i]);
      }
      if (write) emit(c, f);
    }
    if (direct) {
      // A row's 16-byte pieces by neighbouring lanes: whole lines (a thread
      // writing its own row touched 32 lines an instruction, 1.6 us a tile).
      __syncwarp();
      const int pieces = single ? HD / 16 : HD / 8, rows = 32 / pieces;
      const int piece = (single ? t * (HD / 16) : 0) + lane % pieces, r0 = lane / pieces;
      const uint8_t* src = sQ + t * L::kTileBytes + (r & ~31) * (HD * 2);
      for (int i = 0; i < 32; i += rows) {
        const int x = i + r0;
        const long long out = __shfl_sync(0xffffffffu, row.out, x);
        if (__shfl_sync(0xffffffffu, write ? 1 : 0, x))
          *reinterpret_cast<uint4*>(reinterpret_cast<T*>(p.o) + out * HD + piece * 8) =
              *reinterpret_cast<const uint4*>(src + x * (HD * 2) + ((piece ^ (x & 7)) << 4));
      }
    }
    if (write && !(single && t == 1)) {
      if (direct)
        p.lse[row.out] = seen ? (m_ref + __log2f(l_sum)) * 0.69314718055994531f : -INFINITY;
      else
        p.part_ml[part * 128 + r] = make_float2(seen ? m_ref : -INFINITY, l_sum);
    }
    tc_fence_before();
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 8) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// Joins the partial results of every row: those of the key splits above and,
// behind a shared prefix, those of the splits of the sequence's own keys
// (own_o [row][own_S][d], own_ml [row][own_S]).  A block takes 1024 / d
// consecutive rows of a row tile: thread = (row, 4 features), rows fastest, so
// that a warp reads 128 bytes of each split's [d / 4][128] block and 64 of each
// own row.
struct PagedMergeParams {
  PagedParams p;
  const float* own_o;   // nullptr: none
  const float* own_ml;
  int own_S;
};

template <int HD, bool BF16>
__global__ void __launch_bounds__(256) fa_paged_merge_kernel(const __grid_constant__ PagedMergeParams a) {
  using T = typename std::conditional<BF16, __nv_bfloat16, __half>::type;
  const PagedParams& p = a.p;
  constexpr int kRows = 1024 / HD;  // rows of a block: 8 or 16
  constexpr int kGroups = 128 / kRows;
  grid_dependency_wait();
  grid_launch_dependents();
  const int tile_id = blockIdx.x / kGroups;
  const int r = (blockIdx.x % kGroups) * kRows + threadIdx.x % kRows, c4 = threadIdx.x / kRows;
  const int owner = tile_id / p.n_tiles, tile = tile_id % p.n_tiles;
  const PagedRow row = paged_row(p, owner, tile, r);
  if (!row.in_tile) return;
  const bool single = tile >= 2 * p.n_pairs;
  const int S = single ? p.S_single : p.S;
  const long long part = (static_cast<long long>(owner) * p.n_tiles + tile) * p.slots;
  const float2* ml = p.part_ml + part * 128 + r;
  const float4* po = p.part_o + (part * (HD / 4) + c4) * 128 + r;
  const float2* ml2 = reinterpret_cast<const float2*>(a.own_ml) + row.out * a.own_S;
  const float4* po2 = reinterpret_cast<const float4*>(a.own_o + row.out * a.own_S * HD) + c4;
  float m = -INFINITY;
#pragma unroll 8
  for (int s = 0; s < S; ++s) m = fmaxf(m, ml[s * 128].x);
#pragma unroll 4
  for (int s = 0; s < a.own_S; ++s) m = fmaxf(m, ml2[s].x);
  // (asked for after the statistics, which do not depend on the lengths)
  const PagedSeq q = paged_seq(p, row.b);
  if (row.t >= q.row_end) return;
  // a maximum of -inf does not say that the row saw nothing: NaN is no maximum
  const float ref = m == -INFINITY ? 0.f : m;
  float l = 0.f;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  auto add = [&](float2 x, const float4* src) {
    const float w = ex2_approx(x.x - ref);  // 0 for an empty split, whose O is 0
    const float4 y = *src;
    l += x.y * w;
    o.x += y.x * w, o.y += y.y * w, o.z += y.z * w, o.w += y.w * w;
  };
#pragma unroll 4
  for (int s = 0; s < S; ++s) add(ml[s * 128], po + static_cast<long long>(s) * (HD / 4) * 128);
#pragma unroll 4
  for (int s = 0; s < a.own_S; ++s) add(ml2[s], po2 + s * (HD / 4));
  const float inv = l != 0.f ? 1.f / l : 0.f;
  uint2 w;
  w.x = pack2<BF16>(o.x * inv, o.y * inv);
  w.y = pack2<BF16>(o.z * inv, o.w * inv);
  *reinterpret_cast<uint2*>(reinterpret_cast<T*>(p.o) + row.out * HD + 4 * c4) = w;
  if (c4 == 0) p.lse[row.out] = l != 0.f ? (m + __log2f(l)) * 0.69314718055994531f : -INFINITY;
}

}  // namespace fa
