// attention_weights: the attention weight that each cached token gets from a chunk's rows, summed over the
// rows and over the query heads of its kv head, and added to what it had.
//
// Mathematics: with the rows' log-sum-exp known, p = exp(scale q . k - lse) needs no other key: a key's sum
// is its own, and nothing is exchanged between keys.
//
// GB300 design: S^T = K Q^T on tcgen05, 128 keys by up to 128 flat query rows (row f is head f mod G of
// query row f / G), so that a tensor memory lane is a key and its thread adds up a row of exponentials
// without a word to other threads.  Up to four key tiles stay in shared memory while the blocks of query
// rows pass by, each tile's scores in 128 columns of their own: while one tile's products run, the
// exponentials of the others are taken.  One or two blocks of rows stay too, and the key tiles pass by.
// Queries that need no change come by TMA, whole query rows a block; over e4m3 and 4 bits bf16 queries are
// turned into fp16 by the warps that turn the keys.  The list of (chunk, kv head, key tile) is cut over the
// SMs by the number of blocks that see each tile: no tile's sum is split, so no order of sums depends on
// the run.
//
// Bound: few rows, HBM (64 sequences of up to 2,048 tokens, one row each, 28 heads over 4, bf16: 20.4 us,
// 0.55 of the measured copy); many rows, the chain of a slot, products - exponentials - products (2,048
// rows over 8,192 keys, 32 heads over 8, f16: 138 us; the products alone take 62, the exponentials 51),
// where SMs with four key tiles work on for a fifth longer than the mean, and shared memory: the products
// read 8 KB each, and two terms a row beside them instead of one cost 29 us.  Over e4m3 and 4 bits 152 and
// 144 us with f16 queries, 260 and 252 with bf16 ones, which the loader warps turn into fp16 and which have
// two terms a row.  64 rows over up to 16,384 keys of 4 bits: 48 us (f16 queries: 38).  Not faster: the slots in halves of 64 rows (206 us where whole ones took 166:
// products of 64 columns read the keys as often).
#include <algorithm>

#include "paged_tiles.cuh"
#include "umma_issue.cuh"

namespace pkv {
namespace {

constexpr int kThreads = 896;
constexpr uint32_t kTmemCols = 512;           // four slots of 128 columns
constexpr int kSlots = 4;
constexpr int kItems = 8;                     // items on their way from the scheduler to the other warps
constexpr int kMaxChunks = 65535;
constexpr int kSeqChunk = 32;                 // chunks per entry of the table of work
constexpr int kReaders = 16 + 8 + 1 + 1;      // warps that read the items: exponentials, loaders, MMA, key tiles by TMA
// Of a key tile beside its blocks: its load takes as long as about two of them.  (With 0, 1, 2, 3 and 4: 20.4, 20.5, 20.3,
// 20.3 and 20.3 us for one row over 64 sequences, 48.6, 48.6, 48.1, 48.1 and 48.1 for 64 rows over four, 138.7, 138.7, 138.7,
// 136.7 and 136.7 for 2,048 rows over one, whose cuts fall on whole tiles.)
constexpr int kTileCost = 2;

struct WeightsParams {
  float* out;
  const float* in;
  float decay;
  const int32_t* rows;
  const uint8_t* q;
  const float* lse;
  const int32_t* cu_q;
  const int32_t* start;
  const uint8_t* k_cache;
  const float* k_scale;
  int num_rows, max_len, num_chunks, total_q, num_heads;
  float scale_log2;
  Divisor group;          // query heads per kv head
  Divisor block;          // flat rows of a block: 128, or as many whole query rows as that holds (queries by TMA)
  bool tma;               // queries by TMA
  PagedCache pc;
};

// Key tiles of a (chunk, kv head) that this CTA works on.
struct Item {
  int seq, h, q0, start;  // chunk, kv head, first query row, its position
  int F, k0, k1, row;     // flat rows (0: no more items), key tiles, row of the weights
};

// A chunk: its rows, or none where there is nothing to do.
struct Chunk {
  int q0, len, start, row;
  unsigned error;
  __device__ __forceinline__ Chunk(const WeightsParams& p, int s) {
    q0 = p.cu_q[s];
    start = p.start[s];
    row = p.rows ? p.rows[s] : s;
    const int64_t n = int64_t(p.cu_q[s + 1]) - q0;
    error = 0;
    if (q0 < 0 || n < 0 || q0 + n > p.total_q || start < 0 ||
        (n > 0 && start + n > (int64_t(p.pc.max_blocks) << p.pc.block_shift)))
      error = PKV_DEVERR_CHUNK;
    else if (n > 0 && row >= p.num_rows)
      error = PKV_DEVERR_SLOT;
    else if (n > 0 && row >= 0 && start + n > p.max_len)
      error = PKV_DEVERR_CONTEXT_LEN;
    len = error || row < 0 ? 0 : int(n);
  }
  __device__ __forceinline__ int tiles() const { return len == 0 ? 0 : (start + len + kTile - 1) / kTile; }
};

// Blocks of F flat rows, and the first that sees key tile t (which some row does).
__device__ __forceinline__ int blocks_of(const WeightsParams& p, int F) { return int(p.block.quotient(F + int(p.block.d) - 1)); }
__device__ __forceinline__ int first_block(const WeightsParams& p, int start, int t) {
  const int rows = t * kTile - start;
  return rows > 0 ? int(p.block.quotient(rows * int(p.group.d))) : 0;
}

// Key tiles that every block sees; the others come after them.
__device__ __forceinline__ int old_tiles(const Chunk& c) { return min(c.tiles(), c.start / kTile + 1); }

// Work of a chunk's kv head.
__device__ __forceinline__ int units_of(const WeightsParams& p, const Chunk& c) {
  if (c.len == 0) return 0;
  const int blocks = blocks_of(p, c.len * int(p.group.d)), n = old_tiles(c);
  int units = n * (blocks + kTileCost);
  for (int t = n; t < c.tiles(); ++t) units += blocks - first_block(p, c.start, t) + kTileCost;
  return units;
}

// The first key tile at or behind `at` units into a chunk's kv head.
__device__ __forceinline__ int tile_at(const WeightsParams& p, const Chunk& c, int64_t at) {
  if (at <= 0) return 0;
  const int blocks = blocks_of(p, c.len * int(p.group.d)), n = old_tiles(c), per = blocks + kTileCost;
  if (at <= int64_t(n) * per) return int((at + per - 1) / per);
  at -= int64_t(n) * per;
  int t = n;
  for (; t < c.tiles() && at > 0; ++t) at -= blocks - first_block(p, c.start, t) + kTileCost;
  return t;
}

template <int D>
struct Cfg {
  static constexpr int kTileBytes = D / 64 * kHalfBytes;
  static constexpr int kSmem = (kSlots + 2) * kTileBytes;    // key tiles, blocks of queries
};

// ---------------------------------------------------------------------------------------
//   warps 0-15 : exponentials and sums, four warps for each slot of scores; a thread per key
//   warps 16-23: the quantised key tiles and the blocks of queries, four warps each for those of even and odd number
//   warp 24    : cuts this CTA's range of the work into items and hands them to the other warps
//   warp 25    : TMEM owner and MMA issuer
//   warp 26    : key tiles of 16-bit caches by TMA
// An item's key tiles are taken in groups of four (the last may be smaller).  A group's steps are its blocks of queries, and
// within a block its tiles; tile x of a group has slot x.  A group of one or two tiles has two or four slots for each tile,
// taken by turns from block to block, and their sums are added at the end.
// One or two blocks stay for all groups; more pass by once for every group.
// ---------------------------------------------------------------------------------------
template <int KV, bool kBF16, int D>
__global__ void __launch_bounds__(kThreads, 1) weights_kernel(const __grid_constant__ CUtensorMap tmk,
                                                              const __grid_constant__ CUtensorMap tmq, const WeightsParams p) {
  using C = Cfg<D>;
  constexpr bool kWide = KV == PKV_F16 || KV == PKV_BF16;    // 16-bit caches
  constexpr bool kMmaBF16 = KV == PKV_BF16;
  extern __shared__ __align__(1024) uint8_t smem[];
  __shared__ __align__(16) int4 items[kItems][2];
  __shared__ __align__(8) uint64_t bar_item[kItems], bar_item_read[kItems];
  // Query block there / not read any more; key tiles likewise; scores there / read; sums of a group there.
  __shared__ __align__(8) uint64_t bar_q[2], bar_q_empty[2], bar_k[kSlots], bar_k_empty[kSlots], bar_s[kSlots], bar_s_free[kSlots],
      bar_sum, bar_drain;
  __shared__ uint32_t tmem_base_sh;
  // [block number mod 8]: (factor, factor, -lse, -lse) of row pairs; queries by TMA have one factor: only
  // -lse of each row.  Block u + 8 is loaded once the products of u + 6 are done; by then those of u + 4 at
  // the latest have waited for the sums of u, or a smaller group has begun, which waits for all.
  __shared__ __align__(16) float row_terms[8][2 * kTile];
  __shared__ float sums[2][kSlots][kTile];
  __shared__ int first_unit[(kMaxChunks + kSeqChunk - 1) / kSeqChunk + 1];
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;   // uniform in the warp

  uint8_t* sK = smem;                                        // [slot][64-dim half][128 rows]
  uint8_t* sQ = smem + kSlots * C::kTileBytes;               // [block mod 2][64-dim half][128 rows]
  if (smem_u32(smem) & 1023u) {                              // the 128-byte swizzle needs 1 KB alignment
    if (threadIdx.x == 0) set_error(p.pc.err, PKV_DEVERR_CHUNK);
    return;
  }
  if (threadIdx.x == 0) {
    if constexpr (kWide) prefetch_tensormap(&tmk);
    if (p.tma) prefetch_tensormap(&tmq);
    for (int i = 0; i < kItems; ++i) {
      mbar_init(&bar_item[i], 1);
      mbar_init(&bar_item_read[i], kReaders);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bar_q[i], 4);
      mbar_init(&bar_q_empty[i], 1);
    }
    for (int i = 0; i < kSlots; ++i) {
      mbar_init(&bar_k[i], kWide ? 1 : 4);
      mbar_init(&bar_k_empty[i], 1);
      mbar_init(&bar_s[i], 1);
      mbar_init(&bar_s_free[i], 4);
    }
    mbar_init(&bar_sum, 16);
    mbar_init(&bar_drain, 1);
    fence_mbar_init();
  }
  if (warp == 25) {
    tmem_alloc(&tmem_base_sh, kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_base_sh;
  griddep_launch_dependents();
  // Only the set-up above may run before the previous kernel on the stream has finished.
  griddep_wait();

  const int G = int(p.group.d), hkv = p.pc.num_kv_heads;
  auto all = [](bool v) -> bool { return __all_sync(0xffffffffu, v); };

  // The units of each kSeqChunk chunks, then their running sums.
  const int tables = (p.num_chunks + kSeqChunk - 1) / kSeqChunk;
  unsigned error = blockIdx.x == 0 && threadIdx.x == 0 && p.cu_q[0] != 0 ? PKV_DEVERR_CHUNK : 0;
  for (int c = warp; c < tables; c += kThreads / 32) {
    const int s = c * kSeqChunk + lane;
    int units = 0;
    if (s < p.num_chunks) {
      const Chunk ch(p, s);
      units = units_of(p, ch);
      if (blockIdx.x == 0) error |= ch.error;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) units += __shfl_xor_sync(0xffffffffu, units, o);
    if (lane == 0) first_unit[c + 1] = units;
  }
  if (error) set_error(p.pc.err, error);
  __syncthreads();
  if (warp == 0) {
    int total = 0;
    for (int c0 = 0; c0 < tables; c0 += 32) {
      int v = c0 + lane < tables ? first_unit[c0 + lane + 1] : 0;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int w = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += w;
      }
      if (c0 + lane < tables) first_unit[c0 + lane + 1] = total + v;
      total += __shfl_sync(0xffffffffu, v, 31);
    }
    if (lane == 0) first_unit[0] = 0;
  }
  __syncthreads();

  auto wait_item = [&](uint32_t i) -> bool { return all(mbar_wait(&bar_item[i % kItems], i / kItems & 1u)); };
  auto read_item = [&](uint32_t i) -> Item {
    const int4 a = items[i % kItems][0], b = items[i % kItems][1];
    return Item{a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
  };
  auto done_reading = [&](uint32_t i) {
    __syncwarp();
    if (lane == 0) mbar_arrive(&bar_item_read[i % kItems]);
  };
  // Calls group(t, nt, b0) for the groups of nt key tiles from t on, which the blocks from b0 on see.
  auto each_group = [&](const Item& it, auto group) -> bool {
    for (int t = it.k0; t < it.k1; t += kSlots) {
      // Blocks that stay are taken from the first on, so that all groups agree on them.
      const int b0 = blocks_of(p, it.F) <= 2 ? 0 : first_block(p, it.start, t);
      if (!group(t, min(kSlots, it.k1 - t), b0)) return false;
    }
    return true;
  };
  const int BR = int(p.block.d);
  bool ok = true;

  if (warp < 16) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 64;");     // 512 * 64 + 256 * 96 + 128 * 56 = 896 * 72
    // ---------------- exponentials and sums ----------------
    const int x = warp >> 2, r = threadIdx.x & 127;          // slot; key of the tile
    const uint32_t tS = tmem + 128 * x + (uint32_t(32 * (warp & 3)) << 16);
    uint32_t steps = 0, merges = 0, qc = 0;                  // of this slot; smaller groups; blocks so far
    for (uint32_t i = 0;; ++i) {
      ok = ok && wait_item(i);
      if (!ok) break;
      const Item it = read_item(i);
      done_reading(i);
      if (it.F == 0) break;
      const int NB = blocks_of(p, it.F);
      const bool stay = NB <= 2;
      const float slog = p.scale_log2 * (!kWide && p.k_scale ? __ldg(p.k_scale + it.h) : 1.f);           // (queries by TMA)
      ok = each_group(it, [&](int t, int nt, int b0) -> bool {
        const int turns = nt == 1 ? 4 : nt == 2 ? 2 : 1;     // slots of a tile
        const int mine = x < nt * turns ? x % nt : -1, turn = x / nt;        // tile of the group; which of its slots
        const int key = (t + max(mine, 0)) * kTile + r;
        float sum = 0.f, lost = 0.f;                         // compensated
        for (int b = b0 + turn; mine >= 0 && b < NB; b += turns, ++steps) {
          const uint32_t use = qc + (b - (stay ? 0 : b0));   // number of the block among all that were loaded
          if (!all(mbar_wait(&bar_s[x], steps & 1u))) return false;
          tc_fence_after();
          const int n = min(BR, it.F - b * BR);
          const int64_t before = (int64_t(key) - it.start) * G - int64_t(b) * BR;   // rows of the block that do not see the key
          const int lo = int(max(int64_t(0), min(before, int64_t(kTile))));
          const bool whole = all(lo == 0 && n % 32 == 0);
          const float* terms = row_terms[use & 7u];
          uint64_t acc0 = pack_f32x2(0.f, 0.f), acc1 = acc0;
          const int chunks = (n + 31) / 32;
#pragma unroll 1
          for (int cc = 0; cc < chunks; ++cc) {
            uint64_t s[16];
            tmem_ld_pairs(tS + 32 * cc, s);
            if (whole && p.tma) {
              const uint64_t sl2 = pack_f32x2(slog, slog);
#pragma unroll
              for (int c = 0; c < 8; ++c) {                  // (every read of shared memory takes from what the products read)
                const float4 f = reinterpret_cast<const float4*>(terms)[8 * cc + c];
                const uint64_t e0 = fma_f32x2(s[2 * c], sl2, pack_f32x2(f.x, f.y)), e1 = fma_f32x2(s[2 * c + 1], sl2, pack_f32x2(f.z, f.w));
                acc0 = add_f32x2(acc0, pack_f32x2(fast_exp2(lo_f32(e0)), fast_exp2(hi_f32(e0))));
                acc1 = add_f32x2(acc1, pack_f32x2(fast_exp2(lo_f32(e1)), fast_exp2(hi_f32(e1))));
              }
            } else if (whole) {
#pragma unroll
              for (int c = 0; c < 16; ++c) {
                const float4 f = reinterpret_cast<const float4*>(terms)[16 * cc + c];
                const uint64_t e = fma_f32x2(s[c], pack_f32x2(f.x, f.y), pack_f32x2(f.z, f.w));
                const uint64_t pe = pack_f32x2(fast_exp2(lo_f32(e)), fast_exp2(hi_f32(e)));
                if (c & 1) acc1 = add_f32x2(acc1, pe);
                else acc0 = add_f32x2(acc0, pe);
              }
            } else {
#pragma unroll
              for (int c = 0; c < 16; ++c) {
                float4 f;
                if (p.tma) {
                  const float2 e = reinterpret_cast<const float2*>(terms)[16 * cc + c];
                  f = make_float4(slog, slog, e.x, e.y);
                } else {
                  f = reinterpret_cast<const float4*>(terms)[16 * cc + c];
                }
                const int c0 = 32 * cc + 2 * c;
                const float e0 = c0 >= lo && c0 < n ? fmaf(lo_f32(s[c]), f.x, f.z) : -INFINITY;
                const float e1 = c0 + 1 >= lo && c0 + 1 < n ? fmaf(hi_f32(s[c]), f.y, f.w) : -INFINITY;
                const uint64_t pe = pack_f32x2(fast_exp2(e0), fast_exp2(e1));
                if (c & 1) acc1 = add_f32x2(acc1, pe);
                else acc0 = add_f32x2(acc0, pe);
              }
            }
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&bar_s_free[x]);        // the next products may overwrite the scores
          const uint64_t acc = add_f32x2(acc0, acc1);
          const float y = lo_f32(acc) + hi_f32(acc) - lost, z = sum + y;
          lost = (z - sum) - y;
          if (!(fabsf(lost) < INFINITY)) lost = 0.f;
          sum = z;
        }
        if (nt < kSlots) {                                   // (of three tiles: no sums to add, but no slot is left behind)
          const int par = merges & 1u;
          sums[par][x][r] = sum - lost;
          __syncwarp();
          if (lane == 0) mbar_arrive(&bar_sum);
          if (!all(mbar_wait(&bar_sum, par))) return false;
          ++merges;
          if (turn == 0 && turns > 1) {
            sum = 0.f;
            lost = 0.f;
            for (int u = 0; u < turns; ++u) sum += sums[par][u * nt + mine][r];
          }
        }
        if (mine >= 0 && turn == 0 && key < it.start + int(p.group.quotient(it.F))) {
          const int64_t at = (int64_t(it.row) * hkv + it.h) * p.max_len + key;
          sum -= lost;
          p.out[at] = p.in && key < it.start ? fmaf(p.decay, p.in[at], sum) : sum;
        }
        if (!stay) qc += NB - b0;
        return true;
      });
      if (stay) qc += NB;
    }
    if (!ok && lane == 0) set_error(p.pc.err, PKV_DEVERR_TIMEOUT);
  } else if (warp < 24) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 96;");
    // ---------------- key tiles and queries ----------------
    const int par = (warp >> 2) & 1, w = warp & 3, tid = threadIdx.x & 127;
    uint32_t kc = 0, qc = 0, li = 0;                         // key tiles, blocks of queries, item of the tile to load
    StoredTile<kWide ? int(PKV_FP8_E4M3) : KV, D> ahead;     // (16-bit caches: not used)
    TableWindow win;
    Item la = {};
    int lt = par;                                            // the next tile to load, of item `la`
    bool more = !kWide;
    auto load_ahead = [&]() -> bool {
      while (more && lt >= la.k1) {
        const int over = lt - la.k1;
        if (la.F > 0) ++li;
        if (!wait_item(li)) return false;
        la = read_item(li);
        more = la.F > 0;
        if (!more) break;
        lt = la.k0 + over;
        const int end = la.start + int(p.group.quotient(la.F));
        win.open(p.pc.tables + int64_t(la.seq) * p.pc.max_blocks, min(p.pc.max_blocks, ((end - 1) >> p.pc.block_shift) + 1));
      }
      if (more) ahead.load(p.k_cache, p.pc, win, la.h, lt, la.start + int(p.group.quotient(la.F)), w, lane);
      lt += 2;
      return true;
    };
    ok = load_ahead();
    for (uint32_t i = 0; ok; ++i) {
      ok = wait_item(i);
      if (!ok) break;
      const Item it = read_item(i);
      if (it.F == 0) {
        done_reading(i);
        break;
      }
      const int NB = blocks_of(p, it.F);
      const bool stay = NB <= 2;
      ok = each_group(it, [&](int t, int nt, int b0) -> bool {
        // Blocks that stay come before the group's first key tile, others behind it.
#pragma unroll 1
        for (int part = 0; part < 2; ++part) {
          if ((part == 0) != stay) {
            for (int u = 0; u < nt; ++u, ++kc) {
              if (kWide || (kc & 1u) != uint32_t(par)) continue;
              const uint32_t st = kc % kSlots, round = kc / kSlots;
              if (!all(round == 0 || mbar_wait(&bar_k_empty[st], (round - 1) & 1u))) return false;
              ahead.store(smem_u32(sK) + st * C::kTileBytes, w, lane);
              fence_proxy_async_smem();
              __syncwarp();
              if (lane == 0) mbar_arrive(&bar_k[st]);
              if (!load_ahead()) return false;
            }
          } else if (!stay || t == it.k0) {
            for (int b = b0; b < NB; ++b, ++qc) {
              if ((qc & 1u) != uint32_t(par)) continue;
              const uint32_t use = qc >> 1;
              float* terms = row_terms[qc & 7u];
              const int n = min(BR, it.F - b * BR);
              const float head_scale = !kWide && p.k_scale ? __ldg(p.k_scale + it.h) : 1.f;
              if (p.tma) {                                       // (a thread per row for its terms)
                const int f = b * BR + tid, row = int(p.group.quotient(f));
                float e = 0.f;
                if (tid < n) e = __ldg(p.lse + (it.q0 + row) * p.num_heads + it.h * G + (f - row * G)) * -1.4426950408889634f;
                if (!all(use == 0 || mbar_wait(&bar_q_empty[par], (use - 1) & 1u))) return false;
                if (tid == 0) {
                  mbar_expect_tx(&bar_q[par], BR * D * 2);
                  for (int d = 0; d < D / 64; ++d)
                    tma_load_3d(sQ + par * C::kTileBytes + d * kHalfBytes, &tmq, &bar_q[par], 64 * d, it.h * G,
                                it.q0 + int(p.group.quotient(b * BR)), l2_policy_evict_last());
                }
                if (tid < n) terms[tid] = e;
                __syncwarp();
                if (lane == 0) mbar_arrive(&bar_q[par]);         // every warp's behind its terms: they may come later than the copy
                continue;
              }
              const bool loaded = load_queries<kBF16, !kWide, D, 128, 4>(smem_u32(sQ) + par * C::kTileBytes, p.q, it.q0, p.num_heads, it.h, p.group, b * BR, n, 1,
                                                  p.scale_log2, head_scale, tid,
                                                  [&] { return all(use == 0 || mbar_wait(&bar_q_empty[par], (use - 1) & 1u)); },
                                                  [&](int i) { return __ldg(p.lse + i) * -1.4426950408889634f; },
                                                  [&](int row, float c, float e) {
                                                    terms[(row >> 1) * 4 + (row & 1)] = c;
                                                    terms[(row >> 1) * 4 + 2 + (row & 1)] = e;
                                                  });
              if (!loaded) return false;
              fence_proxy_async_smem();
              __syncwarp();
              if (lane == 0) mbar_arrive(&bar_q[par]);
            }
          }
        }
        return true;
      });
      done_reading(i);
    }
    if (!ok && lane == 0) set_error(p.pc.err, PKV_DEVERR_TIMEOUT);
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
    if (warp == 24) {
      // ---------------- this CTA's range of the work, item by item ----------------
      const int64_t total = int64_t(hkv) * first_unit[tables];
      const int64_t lo = total * blockIdx.x / gridDim.x, hi = total * (blockIdx.x + 1) / gridDim.x;
      uint32_t i = 0;
      auto put = [&](const Item& it) {
        ok = ok && (i < uint32_t(kItems) || all(mbar_wait(&bar_item_read[i % kItems], (i / kItems - 1) & 1u)));
        if (!ok) return;
        if (lane == 0) {
          items[i % kItems][0] = make_int4(it.seq, it.h, it.q0, it.start);
          items[i % kItems][1] = make_int4(it.F, it.k0, it.k1, it.row);
          mbar_arrive(&bar_item[i % kItems]);
        }
        __syncwarp();
        ++i;
      };
      if (lo < hi) {
        int a = 0, b = tables;                               // hkv first_unit[a] <= lo < hkv first_unit[a + 1]
        while (b - a > 1) {
          const int mid = (a + b) >> 1;
          if (int64_t(hkv) * first_unit[mid] <= lo) a = mid; else b = mid;
        }
        const int s0 = a * kSeqChunk + lane;
        int mine = s0 < p.num_chunks ? units_of(p, Chunk(p, s0)) : 0, sum = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int v = __shfl_up_sync(0xffffffffu, sum, o);
          if (lane >= o) sum += v;
        }
        const int64_t in_table = lo - int64_t(hkv) * first_unit[a];
        const unsigned past = __ballot_sync(0xffffffffu, int64_t(hkv) * sum > in_table);
        const int l = past ? __ffs(past) - 1 : 31;
        const int64_t before = int64_t(hkv) * __shfl_sync(0xffffffffu, sum - mine, l);
        int units = __shfl_sync(0xffffffffu, mine, l);
        int seq = a * kSeqChunk + l;
        int h = int((in_table - before) / max(1, units));
        int64_t pos = lo - (in_table - before) % max(1, units);              // of the (chunk, kv head)'s first unit
        Chunk ch(p, min(seq, p.num_chunks - 1));
        while (past && pos < hi && ok) {
          if (h >= hkv || units == 0) {                      // the next chunk
            h = 0;
            if (++seq >= p.num_chunks) break;
            ch = Chunk(p, seq);
            units = units_of(p, ch);
            continue;
          }
          Item it;
          it.seq = seq;
          it.h = h;
          it.q0 = ch.q0;
          it.start = ch.start;
          it.F = ch.len * G;
          it.k0 = tile_at(p, ch, lo - pos);
          it.k1 = hi < pos + units ? tile_at(p, ch, hi - pos) : ch.tiles();
          it.row = ch.row;
          if (it.k1 > it.k0) put(it);
          pos += units;
          ++h;
        }
      }
      put(Item{});
    } else if (warp == 25) {
      // ---------------- MMA issuer (the whole warp; see mma_ss) ----------------
      const uint32_t lead = elect_one();
      const uint64_t dK = umma_sdesc_sw128(smem_u32(sK), 16, 1024), dQ = umma_sdesc_sw128(smem_u32(sQ), 16, 1024);
      uint32_t kc = 0, qc = 0, parity = 0;                   // key tiles; blocks; by slot: how often its scores were written, mod 2
      uint32_t open = 0;                                     // by slot: whether these are still to be waited for
      auto wait_free = [&](uint32_t slot) -> bool {
        open &= ~(1u << slot);
        return all(mbar_wait(&bar_s_free[slot], (parity >> slot & 1u) ^ 1u));
      };
      for (uint32_t i = 0;; ++i) {
        ok = ok && wait_item(i);
        if (!ok) break;
        const Item it = read_item(i);
        done_reading(i);
        if (it.F == 0) break;
        const int NB = blocks_of(p, it.F);
        const bool stay = NB <= 2;
        ok = each_group(it, [&](int t, int nt, int b0) -> bool {
          const int turns = nt == 1 ? 4 : nt == 2 ? 2 : 1;
          // Every block of a group of four tiles waits for every slot.  A smaller group may leave slots out, whose
          // warps may still read terms that its blocks would overwrite: they end first.  (64 rows over 16,384 keys
          // take 1 % longer by it.  Looking at each block for slots that are six behind took 2,048 rows over 8,192
          // keys from 138 us to 144.)
          for (uint32_t x = 0; nt < kSlots && x < uint32_t(kSlots); ++x)
            if ((open >> x & 1u) && !wait_free(x)) return false;
          for (int b = b0; b < NB; ++b) {
            const uint32_t use = qc + (b - (stay ? 0 : b0)), st = use & 1u;
            if (!all(mbar_wait(&bar_q[st], use >> 1 & 1u))) return false;
            const uint32_t idesc = umma_idesc_f16(kMmaBF16, 128, (min(BR, it.F - b * BR) + 15) & ~15, false, false);
            for (int u = 0; u < nt; ++u) {
              const uint32_t ks = (kc + u) % kSlots, slot = uint32_t((b - b0) % turns * nt + u);
              if (!all(mbar_wait(&bar_k[ks], (kc + u) / kSlots & 1u))) return false;
              if ((open >> slot & 1u) && !wait_free(slot)) return false;
              open |= 1u << slot;
              parity ^= 1u << slot;
              tc_fence_after();
              const uint64_t da = dK + uint32_t(ks * C::kTileBytes / 16), db = dQ + uint32_t(st * C::kTileBytes / 16);
#pragma unroll
              for (int kk = 0; kk < D / 16; ++kk)
                mma_ss(lead, tmem + 128 * slot, da + ((kk >> 2) * kHalfBytes + (kk & 3) * 32) / 16,
                       db + ((kk >> 2) * kHalfBytes + (kk & 3) * 32) / 16, idesc, kk > 0);
              commit(lead, &bar_s[slot]);
              if (b == NB - 1) commit(lead, &bar_k_empty[ks]);
            }
            if (!stay || t + nt >= it.k1) commit(lead, &bar_q_empty[st]);
          }
          kc += nt;
          if (!stay) qc += NB - b0;
          return true;
        });
        if (!ok) break;
        if (stay) qc += NB;
      }
      commit(lead, &bar_drain);                              // no product may be under way when the CTA leaves
      (void)mbar_wait(&bar_drain, 0);
    } else if (warp == 26) {
      // ---------------- key tiles of 16-bit caches ----------------
      const uint64_t pol = l2_policy_evict_first();
      uint32_t kc = 0;
      TableWindow win;
      for (uint32_t i = 0; ok; ++i) {
        ok = wait_item(i);
        if (!ok) break;
        const Item it = read_item(i);
        done_reading(i);
        if (it.F == 0) break;
        if constexpr (kWide) {
          const int end = it.start + int(p.group.quotient(it.F));
          win.open(p.pc.tables + int64_t(it.seq) * p.pc.max_blocks, min(p.pc.max_blocks, ((end - 1) >> p.pc.block_shift) + 1));
          for (int t = it.k0; t < it.k1 && ok; ++t) {
            const uint32_t st = kc % kSlots, round = kc / kSlots;
            ok = all(round == 0 || mbar_wait(&bar_k_empty[st], (round - 1) & 1u));
            if (!ok) break;
            load_tile_16bit<D>(sK + st * C::kTileBytes, &tmk, &bar_k[st], p.pc, win, it.h, t, end, lane, pol);
            ++kc;
          }
        }
      }
      // No copy may be on its way when the CTA leaves.
      if constexpr (kWide) {
        for (uint32_t u = kc < uint32_t(kSlots) ? 0 : kc - kSlots; u < kc; ++u) (void)mbar_wait(&bar_k[u % kSlots], (u / kSlots) & 1u);
      }
    }
    if (!ok && lane == 0) set_error(p.pc.err, PKV_DEVERR_TIMEOUT);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 25) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

template <int KV, bool kBF16, int D>
pkv_status launch(const CUtensorMap& tk, const CUtensorMap& tq, const WeightsParams& prm, cudaStream_t stream) {
  constexpr int smem = Cfg<D>::kSmem;
  auto kern = weights_kernel<KV, kBF16, D>;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess) return PKV_ERR_CUDA;
  return launch_pdl(kern, dim3(num_sms()), dim3(kThreads), smem, stream, tk, tq, prm) == cudaSuccess ? PKV_OK : PKV_ERR_CUDA;
}

}  // namespace
}  // namespace pkv

extern "C" pkv_status pkv_attention_weights(float* out, const float* weights, float decay, int num_rows, int max_len,
                                            const int32_t* rows, const void* q, pkv_dtype q_dtype, const float* lse,
                                            const int32_t* cu_q_lens, const int32_t* q_start_pos, int num_chunks,
                                            int total_q, int num_heads, const void* k_cache,
                                            const pkv_cache_desc* cache, const int32_t* block_tables,
                                            int max_blocks_per_seq, float scale, pkv_stream_t stream) {
  using namespace pkv;
  pkv_status st = check_cache_desc(cache);
  if (st != PKV_OK) return st;
  if (num_chunks < 0 || total_q < 0 || num_heads <= 0 || max_blocks_per_seq < 0 || num_rows < 0 || max_len < 0 ||
      num_heads % cache->num_kv_heads)
    return PKV_ERR_INVALID_ARG;
  if (q_dtype != PKV_F16 && q_dtype != PKV_BF16) return PKV_ERR_INVALID_ARG;
  if (!(scale > 0.f) || scale > kMostScale || !(decay >= 0.f) || decay > 3.4e38f) return PKV_ERR_INVALID_ARG;
  if ((cache->kv_dtype == PKV_F16 || cache->kv_dtype == PKV_BF16) && cache->kv_dtype != q_dtype)
    return PKV_ERR_UNSUPPORTED;
  if (cache->head_dim != 64 && cache->head_dim != 128) return PKV_ERR_UNSUPPORTED;
  if (cache->block_size != 16 && cache->block_size != 32) return PKV_ERR_UNSUPPORTED;
  if (!chunk_work_fits(num_chunks, total_q, num_heads, max_blocks_per_seq, cache)) return PKV_ERR_UNSUPPORTED;
  if (num_chunks == 0 || total_q == 0) return PKV_OK;
  if (!out || !q || !lse || !cu_q_lens || !q_start_pos || !k_cache || !block_tables || max_blocks_per_seq == 0 ||
      num_rows == 0 || max_len == 0)
    return PKV_ERR_INVALID_ARG;
  auto misaligned = [](const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) != 0; };
  if (!aligned16(q) || !aligned16(k_cache) || misaligned(out) || misaligned(weights) || misaligned(lse) ||
      misaligned(rows) || misaligned(cu_q_lens) || misaligned(q_start_pos) || misaligned(block_tables))
    return PKV_ERR_INVALID_ARG;
  if (!on_current_device(q) || !on_current_device(k_cache)) return PKV_ERR_INVALID_ARG;
  unsigned* err = error_word_ptr();
  if (!err) return PKV_ERR_CUDA;
  const bool wide = cache->kv_dtype == PKV_F16 || cache->kv_dtype == PKV_BF16;
  const int G = num_heads / cache->num_kv_heads;
  // bf16 queries over e4m3 and 4 bits are changed on the way; of more than 128 heads a kv head, no block
  // holds a query row.
  const bool tma = (wide || q_dtype == PKV_F16) && G <= kTile;
  const int whole = tma ? kTile / G : 1;                     // query rows of a block
  WeightsParams prm = {.group = Divisor(G), .block = Divisor(tma ? whole * G : kTile)};
  prm.tma = tma;
  prm.out = out;
  prm.in = weights;
  prm.decay = decay;
  prm.rows = rows;
  prm.q = static_cast<const uint8_t*>(q);
  prm.lse = lse;
  prm.cu_q = cu_q_lens;
  prm.start = q_start_pos;
  prm.k_cache = static_cast<const uint8_t*>(k_cache);
  prm.k_scale = cache->k_scale;
  prm.num_rows = num_rows;
  prm.max_len = max_len;
  prm.num_chunks = num_chunks;
  prm.total_q = total_q;
  prm.num_heads = num_heads;
  prm.scale_log2 = scale * 1.4426950408889634f;
  prm.pc.tables = block_tables;
  prm.pc.max_blocks = max_blocks_per_seq;
  prm.pc.num_blocks = cache->num_blocks;
  prm.pc.num_kv_heads = cache->num_kv_heads;
  prm.pc.block_size = cache->block_size;
  prm.pc.block_shift = cache->block_size == 16 ? 4 : 5;
  prm.pc.err = err;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  CUtensorMap tk = {}, tq = {};
  if (tma && !encode_tmap_3d(&tq, CU_TENSOR_MAP_DATA_TYPE_UINT16, q, uint64_t(cache->head_dim), uint64_t(num_heads),
                             uint64_t(total_q), uint64_t(cache->head_dim) * 2, uint64_t(num_heads) * cache->head_dim * 2, 64, G,
                             whole, CU_TENSOR_MAP_SWIZZLE_128B))
    return PKV_ERR_CUDA;
  if (wide) {                                                // boxes of 64 elements by 16 of the pool's rows
    const int64_t pool_rows = int64_t(cache->num_blocks) * cache->num_kv_heads * cache->block_size;
    if (pool_rows >= (int64_t(1) << 31) - 1) return PKV_ERR_UNSUPPORTED;
    if (!encode_tmap_2d(&tk, CU_TENSOR_MAP_DATA_TYPE_UINT16, k_cache, uint64_t(cache->head_dim), uint64_t(pool_rows),
                        uint64_t(cache->head_dim) * 2, 64, 16, CU_TENSOR_MAP_SWIZZLE_128B))
      return PKV_ERR_CUDA;
  }
  const bool d128 = cache->head_dim == 128, bf = q_dtype == PKV_BF16;
  switch (cache->kv_dtype) {
    case PKV_F16: return d128 ? launch<PKV_F16, false, 128>(tk, tq, prm, s) : launch<PKV_F16, false, 64>(tk, tq, prm, s);
    case PKV_BF16: return d128 ? launch<PKV_BF16, true, 128>(tk, tq, prm, s) : launch<PKV_BF16, true, 64>(tk, tq, prm, s);
    case PKV_FP8_E4M3:
      return bf ? (d128 ? launch<PKV_FP8_E4M3, true, 128>(tk, tq, prm, s) : launch<PKV_FP8_E4M3, true, 64>(tk, tq, prm, s))
                : (d128 ? launch<PKV_FP8_E4M3, false, 128>(tk, tq, prm, s) : launch<PKV_FP8_E4M3, false, 64>(tk, tq, prm, s));
    default:
      return bf ? (d128 ? launch<PKV_FP4_E2M1, true, 128>(tk, tq, prm, s) : launch<PKV_FP4_E2M1, true, 64>(tk, tq, prm, s))
                : (d128 ? launch<PKV_FP4_E2M1, false, 128>(tk, tq, prm, s) : launch<PKV_FP4_E2M1, false, 64>(tk, tq, prm, s));
  }
}
