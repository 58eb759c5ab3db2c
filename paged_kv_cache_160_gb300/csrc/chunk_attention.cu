// paged_chunk_attention: causal attention of each sequence's new rows over its paged cache of any type.
//
// Mathematics: row r of a chunk at positions start .. start + L - 1 attends keys 0 .. start + r, in one
// pass over tiles of 128 keys with the running maximum m and sum l of the softmax (in units of log2): P =
// 2^(s c - m), O = O 2^(m_old - m) + P V; out = O / l, lse = (m + log2 l) ln 2.  Parts of a row's keys are
// merged by their m and l.
//
// GB300 design: the query rows of all heads of a kv head are one list of "flat" rows (row f is head f mod G
// of query row f / G), cut into items of up to 256.  S = Q K^T and O += P V run on tcgen05 with S, P and O
// in tensor memory, in two chains A and B so that one chain's softmax overlaps the other's products: of an
// item's two blocks of 128 rows over the same keys, or, for an item of one block, of every other key tile
// (merged within the CTA).  The list of (item, key tile) is cut into one equal range per SM, whatever the
// chunks' lengths: few rows over long histories use every SM, and no SM works on for long after the others.
// Items that several SMs work on are merged by a second kernel.
//   Quantised rows are read from their blocks into registers, turned into fp16 (exact) and stored as
// operands by 16 warps beside the softmax; 16-bit rows come by TMA.
//
// Bound: the chain of a tile, scores - softmax - products, of which two are under way.  A step takes 2,100
// to 2,300 cycles, its products 1,170: the issuer looks at four barriers a step at 200 cycles each, and the
// softmax of a block takes 1,800.  Measured: 8 sequences of 32K to 128K tokens, 8 rows each, 32 heads
// over 8, D 128, 4 bits: 304 us (the bytes take 101), bf16 360 (360); four chunks of 700 to 1,024 rows
// behind 5K to 9K keys, 32 heads over 8: 459 us over e4m3, 432 over 4 bits, 383 over bf16 (0.58 of the
// measured bf16 rate); 512 rows behind 3,584, 28 heads over 4, 4 bits: 63 us; 64 sequences of up to 2,048
// tokens, 4 rows each: 49 us; 4 of up to 37: 12 us.  (Rows read back from a quantised cache and attended as
// plain ones take 358 us in place of 459 and 37 in place of 63, but 82 in place of 49 and 1,092 in place of
// 304: this kernel is for few rows of many or long sequences, and where there is no room for the rows.)
//   Not faster: two softmax threads a row with half the loader warps (578 us over e4m3), an issuer for each
// chain (489), 64 scores per load from tensor memory, asking L2 for tiles a window ahead.  What made the
// first form three times faster, on the 8 long sequences: no loads in flight spilled (959 us -> 491), rolled
// loops in every role (391; unrolled, the warps' instructions came more slowly than they ran), 16 loader
// warps of one tile each in place of 8 (315), loads without branches (300).
#include <algorithm>

#include "paged_tiles.cuh"
#include "umma_issue.cuh"

namespace pkv {
namespace {

constexpr int kThreads = 896;
constexpr uint32_t kTmemCols = 512;           // S_A | S_B | O_A | O_B, 128 columns each
constexpr float kRescaleThreshold = 8.f;      // log2 units
// fp16 exponentials are taken relative to 2^-kHeadroom of the running maximum: up to 2^15, so that their least step, 2^-24,
// is 2^-31 of a row's largest or less.  (Relative to the maximum itself small weights of many keys vanished: 2^17 keys of
// e^-18 each.)  bf16 has the exponent of fp32 and needs none.  Maxima of kLargeScore and more, in log2 units, are followed
// at once: their own rounding is not added to the threshold then, and 2^(7 + half a spacing) stays below 65504 for maxima up
// to 2^28.
constexpr float kHeadroom = 7.f;
constexpr float kLargeScore = 2097152.f;
constexpr int kItems = 8;                     // items on their way from the scheduler to the other warps
constexpr int kItemRows = 2 * kTile;
// Items of so few rows (a warp's) share each row's keys among four warps: 64 sequences of up to 2,048 tokens, 7 or 28 rows
// a kv head, over 4 bits 43.2 and 48.6 us (a warp for all keys: 45.6 and 50.1), bf16 38.0 and 41.9 (39.7 and 43.9), 256
// sequences of 500 to 1,500 over 4 bits 209 (221).  In long walks the four warps' meeting at each tile costs more than it
// gives: 8 of 32K to 128K tokens, 32 rows, over 4 bits 303 us (291), over e4m3 484 (463), over bf16 359 (359).
constexpr int kFewRows = 32;
constexpr int kMaxChunks = 65535;
constexpr int kSeqChunk = 32;                 // chunks per entry of the table of work
constexpr int kReaders = 8 + 16 + 1 + 2;      // warps that read the items: softmax, loaders, MMA, queries
constexpr int kMergeThreads = 256;

struct ChunkParams {
  uint8_t* out;
  float* lse;
  const uint8_t* q;
  const int32_t* cu_q;
  const int32_t* start;
  const uint8_t* k_cache;
  const uint8_t* v_cache;
  const float* k_scale;
  const float* v_scale;
  uint8_t* parts;         // [2 per CTA] of part_bytes: headers first (see Part)
  int part_rows;          // rows that a part has room for
  int num_chunks, total_q, num_heads;
  float scale_log2;
  Divisor group;          // query heads per kv head
  PagedCache pc;
};

// A part of an item's keys that one CTA has worked on, for the merge: rows = 0: there is none.
struct Part {
  int seq, h, f0, rows, t0, t1, tiles, q0;
};
// Two counters, without an index that would put them in memory.
struct Pair {
  uint32_t a = 0, b = 0;
  __device__ __forceinline__ uint32_t operator[](int x) const { return x ? b : a; }
  __device__ __forceinline__ void up(int x) { x ? ++b : ++a; }
};

// What lies behind the headers of all parts: per part float2 ml[part_rows], float o[part_rows][D].
__host__ __device__ __forceinline__ size_t part_head(int rows) { return size_t(rows + 1) / 2 * 16; }
__host__ __device__ __forceinline__ size_t part_bytes(int rows, int D) { return part_head(rows) + size_t(rows) * 4 * D; }

template <int KV, int D>
struct Cfg {
  static constexpr int kTileBytes = D / 64 * kHalfBytes;     // 128 rows of Q, K or V
  static constexpr int kStages = D == 128 ? 2 : 4;           // K and V tiles in shared memory
  static constexpr int kWeightHalf = kFewRows * 128;         // softmax weights of few rows by 64 keys
  static constexpr int kWeights = 2 * kWeightHalf;           // of a chain
  static constexpr int kSmem = 2 * kWeights + (2 + 2 * kStages) * kTileBytes;
};

// An item's part that this CTA works on.
struct Item {
  int seq, h, q0, start;  // chunk, kv head, first query row, its position
  int f0, rows;           // flat rows (rows = 0: no more items)
  int t0, t1;             // key tiles
  int end;                // keys that the item's last row attends
  int masked;             // key tiles from here on are seen only in part by some rows
  int slot;               // -1: all of the item's keys; else the part to leave it in
  __device__ __forceinline__ bool two() const { return rows > kTile; }
  __device__ __forceinline__ bool few() const { return rows <= kFewRows; }
  __device__ __forceinline__ int steps() const { return two() ? 2 * (t1 - t0) : t1 - t0; }
};

// A chunk: its rows, or none where the lengths are inconsistent.
struct Chunk {
  int q0, len, start;
  bool bad;
  __device__ __forceinline__ Chunk(const ChunkParams& p, int s) {
    q0 = p.cu_q[s];
    start = p.start[s];
    const int64_t n = int64_t(p.cu_q[s + 1]) - q0;
    bad = q0 < 0 || n < 0 || q0 + n > p.total_q || start < 0 ||
          (n > 0 && start + n > (int64_t(p.pc.max_blocks) << p.pc.block_shift));
    len = bad ? 0 : int(n);
  }
};

// Key tiles of the item of flat rows f0 .. f0 + rows - 1.
__device__ __forceinline__ int item_end(const Divisor& group, int start, int f0, int rows) {
  return start + int(group.quotient(f0 + rows - 1)) + 1;
}
__device__ __forceinline__ int tiles_of(int end) { return (end + kTile - 1) / kTile; }

// Work of a chunk's kv head: a unit is one block of 128 rows by one key tile.
__device__ __forceinline__ int units_of(const ChunkParams& p, const Chunk& c) {
  const int F = c.len * int(p.group.d);
  int units = 0;
  for (int f0 = 0; f0 < F; f0 += kItemRows) {
    const int rows = min(kItemRows, F - f0);
    units += tiles_of(item_end(p.group, c.start, f0, rows)) * (rows > kTile ? 2 : 1);
  }
  return units;
}

// Adds to elements d0 .. d1 - 1 of a row that this thread has written (out, of out's type, or o, fp32) the
// non-finite values among V[j] of keys j0 .. j1 - 1 of chunk seq, times `scale`.
template <bool kBF16, int D>
__device__ __noinline__ void give_back(const ChunkParams& p, pkv_dtype kv, int seq, int h, int j0, int j1, int d0, int d1,
                                       float scale, uint8_t* out, float* o) {
  for (int j = j0; j < j1; ++j) {
    const int blk = p.pc.tables[int64_t(seq) * p.pc.max_blocks + (j >> p.pc.block_shift)];
    if (unsigned(blk) >= unsigned(p.pc.num_blocks)) continue;
    const int64_t row = (int64_t(blk) * p.pc.num_kv_heads + h) * p.pc.block_size + (j & (p.pc.block_size - 1));
    for (int c = d0 / 2; c < d1 / 2; ++c) {
      float2 f = cache_pair(p.v_cache, kv, D, row, c);
      if (fabsf(f.x) < INFINITY && fabsf(f.y) < INFINITY) continue;
      f.x = fabsf(f.x) < INFINITY ? 0.f : f.x * scale;
      f.y = fabsf(f.y) < INFINITY ? 0.f : f.y * scale;
      if (o) {
        o[2 * c] += f.x;
        o[2 * c + 1] += f.y;
      } else {
        uint32_t* w = reinterpret_cast<uint32_t*>(out) + c;
        const float2 old = unpack2<kBF16>(*w);
        *w = pack2<kBF16>(old.x + f.x, old.y + f.y);
      }
    }
  }
}

// ---------------------------------------------------------------------------------------
//   warps 0-3  : softmax of chain A, warps 4-7: of chain B; a thread per row.  Also the queries of items of two blocks
//   warps 8-23 : the quantised tiles, four warps each for K and V tiles of even and odd number.  (16-bit caches: warp 8 asks
//                for K and warp 9 for V by TMA.)  V tiles that some rows see only in part are looked at: 0 * V must not turn the
//                rows' other keys into NaN.  Values that are not finite become zeros there, and the rows that do see them get
//                them back at the end
//   warp 24    : cuts this CTA's range of the work into items and hands them to the other warps
//   warp 25    : TMEM owner and MMA issuer, in the order S(0) S(1) | PV(n) S(n + 2) ..., step n in chain n mod 2
//   warps 26-27: queries of items of one block, in the two query areas by turns, ahead of the products
// Every barrier's phases are counted over all items by each of its users.
// ---------------------------------------------------------------------------------------
template <int KV, bool kBF16, int D>
__global__ void __launch_bounds__(kThreads, 1)
    chunk_kernel(const __grid_constant__ CUtensorMap tmk, const __grid_constant__ CUtensorMap tmv, const ChunkParams p) {
  using C = Cfg<KV, D>;
  constexpr bool kWide = KV == PKV_F16 || KV == PKV_BF16;    // 16-bit caches
  constexpr bool kMmaBF16 = KV == PKV_BF16;
  constexpr float kBelow = kMmaBF16 ? 0.f : kHeadroom;
  auto grows = [](float mt, float m) -> bool {
    return mt > m + (kMmaBF16 || fabsf(mt) < kLargeScore ? kRescaleThreshold : 0.f);
  };
  constexpr int kStages = C::kStages;
  extern __shared__ __align__(1024) uint8_t smem[];
  __shared__ __align__(16) int items[kItems][12];
  __shared__ __align__(8) uint64_t bar_item[kItems], bar_item_read[kItems];
  // Q area filled / no product reads it any more; K, V tiles likewise (V: looked at); S_x ready; P_x
  // ready; PV_x done; O read; both chains' maxima and sums there.
  __shared__ __align__(8) uint64_t bar_q[2], bar_q_empty[2], bar_k_full[kStages], bar_k_empty[kStages], bar_v_full[kStages],
      bar_v_seen[kStages], bar_v_empty[kStages], bar_s_full[2], bar_p_full[2], bar_pv_done[2], bar_o_free, bar_ml,
      bar_peak[2], bar_drain;
  __shared__ uint32_t tmem_base_sh;
  __shared__ float factor[2][2][kTile];                      // [query area][use mod 2][row]: products to scores in log2 units
  __shared__ __align__(8) float2 chain_ml[2][2][kTile];      // [item parity][chain][row]
  __shared__ float peak[2][2][4][kFewRows];                  // [chain][step mod 2][quarter of the keys][row]: largest scores
  __shared__ int masked_item[2 * kItems];                    // by item number modulo that: the last such item that non-finite
                                                             // values were taken out for, + 1
  __shared__ int first_unit[(kMaxChunks + kSeqChunk - 1) / kSeqChunk + 1];
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;   // uniform in the warp

  // Weights of few rows come first: as an operand of 128 rows they reach into the queries, whose rows
  // count for nothing.
  uint8_t* sP = smem;                                        // [chain][64-key half][32 rows]
  uint8_t* sQ = smem + 2 * C::kWeights;                      // [area][64-dim half][128 rows]
  uint8_t* sK = sQ + 2 * C::kTileBytes;                      // [stage][64-dim half][128 rows]
  uint8_t* sV = sK + kStages * C::kTileBytes;
  if (smem_u32(smem) & 1023u) {                              // the 128-byte swizzle needs 1 KB alignment
    if (threadIdx.x == 0) set_error(p.pc.err, PKV_DEVERR_CHUNK);
    return;
  }
  if (threadIdx.x == 0) {
    if constexpr (kWide) {
      prefetch_tensormap(&tmk);
      prefetch_tensormap(&tmv);
    }
    for (int i = 0; i < 2 * kItems; ++i) masked_item[i] = 0;
    for (int i = 0; i < kItems; ++i) {
      mbar_init(&bar_item[i], 1);
      mbar_init(&bar_item_read[i], kReaders);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bar_q[i], 6);                               // the warps of a chain and the two for the queries
      mbar_init(&bar_q_empty[i], 1);
      mbar_init(&bar_s_full[i], 1);
      mbar_init(&bar_p_full[i], 4);                          // one arrival per softmax warp
      mbar_init(&bar_pv_done[i], 1);
      mbar_init(&bar_peak[i], 4);
    }
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&bar_k_full[i], kWide ? 1 : 4);
      mbar_init(&bar_k_empty[i], 1);
      mbar_init(&bar_v_full[i], 1);
      mbar_init(&bar_v_seen[i], 4);
      mbar_init(&bar_v_empty[i], 1);
    }
    mbar_init(&bar_o_free, 8);
    mbar_init(&bar_ml, 8);
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
  griddep_launch_dependents();                               // the merge waits for this kernel's end
  // Only the set-up above may run before the previous kernel on the stream has finished.
  griddep_wait();

  const int G = int(p.group.d), hkv = p.pc.num_kv_heads;
  auto all = [](bool v) -> bool { return __all_sync(0xffffffffu, v); };

  // The units of each kSeqChunk chunks, then their running sums.
  const int tables = (p.num_chunks + kSeqChunk - 1) / kSeqChunk;
  bool bad = blockIdx.x == 0 && threadIdx.x == 0 && p.cu_q[0] != 0;
  for (int c = warp; c < tables; c += kThreads / 32) {
    const int s = c * kSeqChunk + lane;
    int units = 0;
    if (s < p.num_chunks) {
      const Chunk ch(p, s);
      units = units_of(p, ch);
      bad |= blockIdx.x == 0 && ch.bad;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) units += __shfl_xor_sync(0xffffffffu, units, o);
    if (lane == 0) first_unit[c + 1] = units;
  }
  if (bad) set_error(p.pc.err, PKV_DEVERR_CHUNK);
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

  auto read_item = [&](uint32_t i) -> Item {
    const int4* w = reinterpret_cast<const int4*>(items[i % kItems]);
    const int4 a = w[0], b = w[1], c = w[2];
    return Item{a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w, c.x, c.y, c.z};
  };
  auto wait_item = [&](uint32_t i) -> bool { return all(mbar_wait(&bar_item[i % kItems], i / kItems & 1u)); };
  auto done_reading = [&](uint32_t i) {
    __syncwarp();
    if (lane == 0) mbar_arrive(&bar_item_read[i % kItems]);
  };
  bool ok = true;

  if (warp < 8) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 96;");     // 256 * 96 + 512 * 64 + 128 * 56 = 896 * 72
    // ---------------- softmax and output: a thread per row ----------------
    const int x = warp >> 2, quarter = warp & 3, r = 32 * quarter + lane;    // TMEM lane == row of the block
    const uint32_t lane_off = uint32_t(32 * quarter) << 16;
    const uint32_t tS = tmem + 128 * x + lane_off, tO = tmem + 256 + lane_off;
    uint32_t steps = 0, turn = 0, merges = 0, peaks = 0;     // this chain's steps; items of one block; steps of few rows
    Pair uses;                                               // of the query areas
    // The item before this one is written after this one's queries (of two blocks) are under way.
    Item it = {};
    bool two = false, few = false, busy = false;
    int rows = 0, f = 0, qrow = 0, keys = 0, nx = 0;
    float m = 0.f, l = 0.f;
    for (uint32_t n = 0;; ++n) {
      ok = ok && wait_item(n);
      if (!ok) break;
      const Item next = read_item(n);
      done_reading(n);
      if (next.two()) {
        float* fac = factor[x][uses[x] & 1u];
        ok = load_queries<kBF16, !kWide, D, 128, 4>(smem_u32(sQ) + x * C::kTileBytes, p.q, next.q0, p.num_heads, next.h, p.group,
                                            next.f0 + kTile * x, x == 0 ? kTile : next.rows - kTile, 1, p.scale_log2,
                                            !kWide && p.k_scale ? __ldg(p.k_scale + next.h) : 1.f, int(threadIdx.x & 127),
                                            [&] { return all(uses[x] == 0 || mbar_wait(&bar_q_empty[x], (uses[x] - 1) & 1u)); },
                                            [](int) { return 0.f; }, [&](int row, float c, float) { fac[row] = c; });
        if (!ok) break;
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar_q[x]);
      }
      if (n > 0) {
        // ---------------- output of item n - 1 ----------------
        const uint32_t i = n - 1;
        ok = ok && (nx == 0 || all(mbar_wait(&bar_pv_done[x], (steps - 1) & 1u)));
        if (!ok) break;
        // m = -inf stands for no keys; a row whose scores are all NaN has some.
        if (m == -INFINITY && l != 0.f) m = 0.f;
        float2 ml0 = make_float2(m, l), ml1 = make_float2(-INFINITY, 0.f);     // of the chains that hold this row
        if (!two) {
          const int par = merges & 1u;
          tc_fence_after();
          tc_fence_before();
          chain_ml[par][x][r] = make_float2(m, l);
          __syncwarp();
          if (lane == 0) mbar_arrive(&bar_ml);
          ok = all(mbar_wait(&bar_ml, par));
          if (!ok) break;
          ++merges;
          ml0 = chain_ml[par][0][r];
          ml1 = chain_ml[par][1][r];
          if (few && quarter == 0) {                         // the sums of the other quarters' keys
            for (int c = 1; c < 4; ++c) {
              ml0.y += chain_ml[par][0][32 * c + lane].y;
              ml1.y += chain_ml[par][1][32 * c + lane].y;
            }
            if (ml0.x == -INFINITY && ml0.y != 0.f) ml0.x = 0.f;
            if (ml1.x == -INFINITY && ml1.y != 0.f) ml1.x = 0.f;
          }
        }
        tc_fence_after();
        const float top = fmaxf(ml0.x, ml1.x);
        const bool have0 = ml0.x != -INFINITY, have1 = ml1.x != -INFINITY;
        float w0 = have0 ? fast_exp2(ml0.x - top) : 0.f, w1 = have1 ? fast_exp2(ml1.x - top) : 0.f;
        const float sum = w0 * ml0.y + w1 * ml1.y;
        const bool taken = *static_cast<volatile int*>(&masked_item[i % (2 * kItems)]) == int(i) + 1;
        const int64_t unit = (int64_t(it.q0) + qrow) * p.num_heads + int64_t(it.h) * G + (f - qrow * G);   // row of out
        const float vs = !kWide && p.v_scale ? __ldg(p.v_scale + it.h) : 1.f;
        const float scale = it.slot >= 0 ? 1.f : sum == 0.f ? 0.f : vs / sum;
        w0 *= scale;
        w1 *= scale;
        float* part_o = nullptr;
        if (it.slot >= 0) {
          uint8_t* body = p.parts + size_t(gridDim.x) * 2 * sizeof(Part) + size_t(it.slot) * part_bytes(p.part_rows, D);
          const int pr = (two ? kTile * x : 0) + r;
          part_o = reinterpret_cast<float*>(body + part_head(p.part_rows)) + size_t(pr) * D;
          if (r < rows && (two || x == 0)) reinterpret_cast<float2*>(body)[pr] = make_float2(top, sum);
        } else if (p.lse && r < rows && (two || x == 0)) {
          p.lse[unit] = (top + log2f(sum)) * 0.6931471805599453f;
        }
        // Items of one block: each chain writes half of the elements, from both chains' O.
        const int c0 = two ? 0 : x * (D / 64), c1 = two ? D / 32 : c0 + D / 64;
        if (busy) {
          for (int cc = c0; cc < c1; ++cc) {
            float v[32];
            if (two) {
              tmem_ld32(tO + 128 * x + 32 * cc, v);
              tmem_wait_ld();
#pragma unroll
              for (int c = 0; c < 32; ++c) v[c] = have0 ? v[c] * w0 : 0.f;
            } else {
              float b[32];
              tmem_ld32(tO + 32 * cc, v);
              tmem_ld32(tO + 128 + 32 * cc, b);
              tmem_wait_ld();
#pragma unroll
              for (int c = 0; c < 32; ++c) v[c] = (have0 ? v[c] * w0 : 0.f) + (have1 ? b[c] * w1 : 0.f);
            }
            if (r < rows) {
              if (it.slot >= 0) {
#pragma unroll
                for (int c = 0; c < 8; ++c)
                  reinterpret_cast<float4*>(part_o)[8 * cc + c] = make_float4(v[4 * c], v[4 * c + 1], v[4 * c + 2], v[4 * c + 3]);
              } else {
                uint4* dst = reinterpret_cast<uint4*>(p.out + unit * (2 * D) + 64 * cc);
#pragma unroll
                for (int c = 0; c < 4; ++c)
                  dst[c] = make_uint4(pack2<kBF16>(v[8 * c], v[8 * c + 1]), pack2<kBF16>(v[8 * c + 2], v[8 * c + 3]),
                                      pack2<kBF16>(v[8 * c + 4], v[8 * c + 5]), pack2<kBF16>(v[8 * c + 6], v[8 * c + 7]));
              }
            }
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar_o_free);
        if (taken && r < rows)
          give_back<kBF16, D>(p, pkv_dtype(KV), it.seq, it.h, max(it.masked, it.t0) * kTile, min(keys, it.t1 * kTile), 32 * c0, 32 * c1,
                              it.slot < 0 ? vs : 1.f, p.out + unit * (2 * D), part_o);
      }
      if (next.rows == 0) break;
      it = next;
      two = it.two();
      const int tiles = it.t1 - it.t0;
      nx = two ? tiles : (tiles + 1 - x) / 2;
      rows = two ? (x == 0 ? kTile : it.rows - kTile) : it.rows;             // of this chain's block
      few = it.few();
      busy = 32 * quarter < rows;                            // some row of this warp exists (of O: few rows are warp 0's)
      const int rr = min(few ? lane : r, rows - 1);
      f = it.f0 + (two ? kTile * x : 0) + rr;
      qrow = int(p.group.quotient(f));
      keys = it.start + qrow + 1;
      const int area = two ? x : int(turn & 1u);
      const float* fac = &factor[area][uses[area] & 1u][rr];
      if (two) {
        uses.up(0);
        uses.up(1);
      } else {
        uses.up(area);
        ++turn;
      }
      m = -INFINITY;
      l = 0.f;
      float slog = 0.f;
      for (int k = 0; k < nx && ok; ++k) {
        const int tile = it.t0 + (two ? k : 2 * k + x);
        // Waiting for the last PV on every step keeps that barrier at most one phase ahead of this wait.
        ok = all(mbar_wait(&bar_s_full[x], (steps + k) & 1u) && (k == 0 || mbar_wait(&bar_pv_done[x], (steps + k - 1) & 1u)));
        if (!ok) break;
        tc_fence_after();
        if (k == 0) slog = *fac;
        const int lim = keys - tile * kTile;                 // keys 0 .. lim - 1 are attended
        if (few) {
          // Every quarter of the lanes has a copy of the rows' scores; its warp takes a quarter
          // of the keys.  One warp for all of a row's keys took 2400 cycles a tile, on one of the
          // SM's four schedulers.
          float s[32];
          tmem_ld32(tS + 32 * quarter, s);
          tmem_wait_ld();
          if (__any_sync(0xffffffffu, lim < 32 * (quarter + 1))) {
#pragma unroll
            for (int c = 0; c < 32; ++c) s[c] = 32 * quarter + c < lim ? s[c] : -INFINITY;
          }
          float c4[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
          for (int c = 4; c < 32; c += 8) {
#pragma unroll
            for (int u = 0; u < 4; ++u)
              if (c + 2 * u + 1 < 32) c4[u] = fmax3(c4[u], s[c + 2 * u], s[c + 2 * u + 1]);
          }
          float(*pk)[kFewRows] = peak[x][peaks & 1u];
          pk[quarter][lane] = fmaxf(fmaxf(c4[0], c4[1]), fmaxf(c4[2], c4[3]));
          __syncwarp();
          if (lane == 0) mbar_arrive(&bar_peak[x]);
          ok = all(mbar_wait(&bar_peak[x], peaks & 1u));
          if (!ok) break;
          ++peaks;
          const float mt = fmaxf(fmaxf(pk[0][lane], pk[1][lane]), fmaxf(pk[2][lane], pk[3][lane])) * slog - kBelow;
          const bool grow = grows(mt, m);                    // (the same in all four warps)
          const float m_prev = m;
          if (grow) m = mt;
          const float mu = m == -INFINITY ? 0.f : m;
          const uint64_t sl2 = pack_f32x2(slog, slog), nm2 = pack_f32x2(-mu, -mu);
          uint64_t acc0 = pack_f32x2(0.f, 0.f), acc1 = acc0;
          const uint32_t row = smem_u32(sP) + x * C::kWeights + (quarter >> 1) * C::kWeightHalf;
#pragma unroll
          for (int g = 0; g < 4; ++g) {                      // 8 keys: 16 bytes
            uint32_t w[4];
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              const uint64_t x2 = fma_f32x2(pack_f32x2(s[8 * g + 2 * c], s[8 * g + 2 * c + 1]), sl2, nm2);
              const float pa = fast_exp2(lo_f32(x2)), pb = fast_exp2(hi_f32(x2));
              const uint64_t p2 = pack_f32x2(pa, pb);
              if (c & 1) acc1 = add_f32x2(acc1, p2);
              else acc0 = add_f32x2(acc0, p2);
              w[c] = pack2<kMmaBF16>(pa, pb);
            }
            sts128(row + swz128(lane, 4 * (quarter & 1) + g), w[0], w[1], w[2], w[3]);
          }
          if (__any_sync(0xffffffffu, grow && k >= 1)) {
            const float alpha = (grow && m_prev != -INFINITY) ? fast_exp2(m_prev - m) : 1.f;
            if (quarter == 0) {                              // the rows of O
#pragma unroll 1
              for (int cc = 0; cc < D / 32; ++cc) {
                float v[32];
                tmem_ld32(tO + 128 * x + 32 * cc, v);
                tmem_wait_ld();
#pragma unroll
                for (int c = 0; c < 32; ++c) v[c] *= alpha;
                tmem_st32(tO + 128 * x + 32 * cc, v);
              }
              tmem_wait_st();
            }
            if (grow) l *= alpha;
          }
          const uint64_t acc = add_f32x2(acc0, acc1);
          l += lo_f32(acc) + hi_f32(acc);
          fence_proxy_async_smem();                          // the weights, to the tensor cores
        } else if (busy) {
          if (__any_sync(0xffffffffu, lim < kTile)) {        // the others' scores: -inf
#pragma unroll 1
            for (int cc = 0; cc < 4; ++cc) {
              float s[32];
              tmem_ld32(tS + 32 * cc, s);
              tmem_wait_ld();
#pragma unroll
              for (int c = 0; c < 32; ++c) s[c] = 32 * cc + c < lim ? s[c] : -INFINITY;
              tmem_st32(tS + 32 * cc, s);
            }
            tmem_wait_st();
          }
          float mt = -INFINITY;
#pragma unroll 1
          for (int cc = 0; cc < 4; ++cc) {
            float s[32];
            tmem_ld32(tS + 32 * cc, s);
            tmem_wait_ld();
            float c4[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
            for (int c = 4; c < 32; c += 8) {
#pragma unroll
              for (int u = 0; u < 4; ++u)
                if (c + 2 * u + 1 < 32) c4[u] = fmax3(c4[u], s[c + 2 * u], s[c + 2 * u + 1]);
            }
            mt = fmaxf(mt, fmaxf(fmaxf(c4[0], c4[1]), fmaxf(c4[2], c4[3])));
          }
          mt = mt * slog - kBelow;                           // (slog > 0)
          const bool grow = grows(mt, m);                    // also true for the first keys
          const float m_prev = m;
          if (grow) m = mt;
          // P over S (keys 2e, 2e + 1 in column e).  A row without keys so far has m = -inf and every
          // s = -inf: P = 0 then.
          const float mu = m == -INFINITY ? 0.f : m;
          const uint64_t sl2 = pack_f32x2(slog, slog), nm2 = pack_f32x2(-mu, -mu);
          uint64_t acc0 = pack_f32x2(0.f, 0.f), acc1 = acc0;
#pragma unroll 1
          for (int cc = 0; cc < 4; ++cc) {
            float s[32];
            tmem_ld32(tS + 32 * cc, s);
            tmem_wait_ld();
            uint32_t w[16];
#pragma unroll
            for (int c = 0; c < 16; ++c) {
              const uint64_t x2 = fma_f32x2(pack_f32x2(s[2 * c], s[2 * c + 1]), sl2, nm2);
              const float pa = fast_exp2(lo_f32(x2)), pb = fast_exp2(hi_f32(x2));
              const uint64_t p2 = pack_f32x2(pa, pb);
              if (c & 1) acc1 = add_f32x2(acc1, p2);
              else acc0 = add_f32x2(acc0, p2);
              w[c] = pack2<kMmaBF16>(pa, pb);
            }
            tmem_st16u(tS + 16 * cc, w);
          }
          if (__any_sync(0xffffffffu, grow && k >= 1)) {     // rescale this row of O
            const float alpha = (grow && m_prev != -INFINITY) ? fast_exp2(m_prev - m) : 1.f;
#pragma unroll 1
            for (int cc = 0; cc < D / 32; ++cc) {
              float v[32];
              tmem_ld32(tO + 128 * x + 32 * cc, v);
              tmem_wait_ld();
#pragma unroll
              for (int c = 0; c < 32; ++c) v[c] *= alpha;
              tmem_st32(tO + 128 * x + 32 * cc, v);
            }
            if (grow) l *= alpha;
          }
          tmem_wait_st();
          const uint64_t acc = add_f32x2(acc0, acc1);
          l += lo_f32(acc) + hi_f32(acc);
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar_p_full[x]);
      }
      steps += nx;
    }
  } else if (warp < 24) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 64;");
    // ---------------- K and V tiles ----------------
    const bool is_v = (warp >> 2 & 1) != 0;
    const int w = warp & 3, par = warp >= 16;                // quantised: tiles of one parity
    if constexpr (kWide) {
      const uint64_t pol = l2_policy_evict_last();
      const int tid = threadIdx.x & 127;
      uint32_t kt = 0;                                       // tiles
      TableWindow win;
      for (uint32_t i = 0; ok; ++i) {
        ok = wait_item(i);
        if (!ok) break;
        const Item it = read_item(i);
        done_reading(i);
        if (it.rows == 0) break;
        win.open(p.pc.tables + int64_t(it.seq) * p.pc.max_blocks, min(p.pc.max_blocks, ((it.end - 1) >> p.pc.block_shift) + 1));
        for (int t = it.t0; t < it.t1 && ok; ++t, ++kt) {
          const uint32_t st = kt % kStages, n = kt / kStages;
          if (!is_v) {
            if (w > 1 || par) continue;
            ok = all(n == 0 || mbar_wait(w == 0 ? &bar_k_empty[st] : &bar_v_empty[st], (n - 1) & 1u));
            if (!ok) break;
            load_tile_16bit<D>((w == 0 ? sK : sV) + st * C::kTileBytes, w == 0 ? &tmk : &tmv,
                               w == 0 ? &bar_k_full[st] : &bar_v_full[st], p.pc, win, it.h, t, it.end, lane, pol);
          } else if (!par) {
            ok = all(mbar_wait(&bar_v_full[st], n & 1u));
            if (!ok) break;
            if (t >= it.masked) {
              const uint32_t base = smem_u32(sV) + st * C::kTileBytes;
              if (t * kTile + tid >= it.end) {
#pragma unroll
                for (int c = 0; c < D / 8; ++c) sts128(operand_at(base, tid, c), 0u, 0u, 0u, 0u);
              } else if (make_row_finite<kMmaBF16, D>(base, tid)) {
                *static_cast<volatile int*>(&masked_item[i % (2 * kItems)]) = int(i) + 1;
              }
              fence_proxy_async_smem();                      // the tile, to the tensor cores
              __syncwarp();
            }
            if (lane == 0) mbar_arrive(&bar_v_seen[st]);
          }
        }
      }
      if (!is_v && w <= 1 && !par) {                                 // no copy may be on its way when the CTA leaves
        for (uint32_t u = kt < uint32_t(kStages) ? 0 : kt - kStages; u < kt; ++u)
          (void)mbar_wait(w == 0 ? &bar_k_full[u % kStages] : &bar_v_full[u % kStages], (u / kStages) & 1u);
      }
    } else {
      // A tile is on its way in registers while the one before it is turned (la: the item of the tile
      // to load, it: of the tile to store).  Loops that stay small: with two tiles' registers and
      // code in each of 8 warps, instructions were fetched more slowly than they ran (8 sequences of
      // 32K to 128K tokens: 391 us).
      StoredTile<KV, D> ahead;
      TableWindow win;
      const uint8_t* cache = is_v ? p.v_cache : p.k_cache;
      uint32_t li = 0, i = 0, kt = par;
      Item la = {}, it = {};
      int lt = par, t = par;                                 // their next tiles
      bool more = true;
      while (true) {
        if (kt >= 2) {                                       // store tile kt - 2
          while (t >= it.t1) {                               // (first: 0 >= 0)
            const int over = t - it.t1;
            if (it.rows > 0) done_reading(i++);
            ok = ok && wait_item(i);
            if (!ok) break;
            it = read_item(i);
            if (it.rows == 0) break;
            t = it.t0 + over;
          }
          if (!ok || it.rows == 0) break;
          const uint32_t n = kt - 2, st = n % kStages, round = n / kStages;
          ok = all(round == 0 || mbar_wait(is_v ? &bar_v_empty[st] : &bar_k_empty[st], (round - 1) & 1u));
          if (!ok) break;
          const uint32_t base = smem_u32(is_v ? sV : sK) + st * C::kTileBytes;
          ahead.store(base, w, lane);
          if (is_v && t >= it.masked) {
            __syncwarp();                                    // a row's lanes are of one warp
            if (make_row_finite<false, D>(base, StoredTile<KV, D>::row_of_lane(w, lane)))
              *static_cast<volatile int*>(&masked_item[i % (2 * kItems)]) = int(i) + 1;
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(is_v ? &bar_v_seen[st] : &bar_k_full[st]);
          t += 2;
        }
        while (more && lt >= la.t1) {
          const int over = lt - la.t1;
          if (la.rows > 0) ++li;
          ok = wait_item(li);
          if (!ok) break;
          la = read_item(li);
          more = la.rows > 0;
          if (!more) break;
          lt = la.t0 + over;
          win.open(p.pc.tables + int64_t(la.seq) * p.pc.max_blocks, min(p.pc.max_blocks, ((la.end - 1) >> p.pc.block_shift) + 1));
        }
        if (!ok) break;
        if (more) ahead.load(cache, p.pc, win, la.h, lt, la.end, w, lane);
        lt += 2;
        kt += 2;
      }
      if (ok && it.rows == 0) done_reading(i);
    }
    if (!ok && lane == 0) set_error(p.pc.err, PKV_DEVERR_TIMEOUT);
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
    if (warp == 24) {
      // ---------------- this CTA's range of the work, item by item ----------------
      const int64_t total = int64_t(hkv) * first_unit[tables];
      const int64_t lo = total * blockIdx.x / gridDim.x, hi = total * (blockIdx.x + 1) / gridDim.x;
      Part parts[2] = {};
      uint32_t i = 0;
      auto put = [&](const Item& it) {
        ok = ok && (i < uint32_t(kItems) || all(mbar_wait(&bar_item_read[i % kItems], (i / kItems - 1) & 1u)));
        if (!ok) return;
        if (lane == 0) {
          int4* w = reinterpret_cast<int4*>(items[i % kItems]);
          w[0] = make_int4(it.seq, it.h, it.q0, it.start);
          w[1] = make_int4(it.f0, it.rows, it.t0, it.t1);
          w[2] = make_int4(it.end, it.masked, it.slot, 0);
          mbar_arrive(&bar_item[i % kItems]);
        }
        __syncwarp();
        ++i;
      };
      if (lo < hi) {
        int a = 0, b = tables;                                 // hkv first_unit[a] <= lo < hkv first_unit[a + 1]
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
        const int units = max(1, __shfl_sync(0xffffffffu, mine, l));
        int seq = a * kSeqChunk + l;
        int h = int((in_table - before) / units);
        int64_t pos = lo - (in_table - before) % units;        // of the current item's first unit
        Chunk ch(p, min(seq, p.num_chunks - 1));
        int f0 = 0;
        while (past && seq < p.num_chunks && pos < hi && ok) {
          const int F = ch.len * G;
          if (h >= hkv || F == 0) {                            // the next chunk
            h = 0;
            f0 = 0;
            if (++seq < p.num_chunks) ch = Chunk(p, seq);
            continue;
          }
          if (f0 >= F) {
            f0 = 0;
            ++h;
            continue;
          }
          Item it;
          it.seq = seq;
          it.h = h;
          it.q0 = ch.q0;
          it.start = ch.start;
          it.f0 = f0;
          it.rows = min(kItemRows, F - f0);
          it.end = item_end(p.group, ch.start, f0, it.rows);
          it.masked = (ch.start + int(p.group.quotient(f0)) + 1) / kTile;
          const int tiles = tiles_of(it.end), cost = it.two() ? 2 : 1;
          const int64_t next = pos + int64_t(tiles) * cost;
          if (next > lo) {
            it.t0 = lo > pos ? int((lo - pos + cost - 1) / cost) : 0;
            it.t1 = hi < next ? int((hi - pos + cost - 1) / cost) : tiles;
            if (it.t1 > it.t0) {
              const int which = pos > lo;
              it.slot = it.t0 == 0 && it.t1 == tiles ? -1 : int(2 * blockIdx.x + which);
              if (it.slot >= 0) parts[which] = Part{seq, h, f0, it.rows, it.t0, it.t1, tiles, ch.q0};
              put(it);
            }
          }
          pos = next;
          f0 += kItemRows;
        }
      }
      if (lane < 2) reinterpret_cast<Part*>(p.parts)[2 * blockIdx.x + lane] = lane ? parts[1] : parts[0];
      put(Item{});
      if (!ok && lane == 0) set_error(p.pc.err, PKV_DEVERR_TIMEOUT);
    } else if (warp == 25) {
      // ---------------- MMA issuer (the whole warp; see mma_ss) ----------------
      const uint32_t lead = elect_one();
      constexpr uint32_t idesc_s = umma_idesc_f16(kMmaBF16, 128, 128, false, false);
      constexpr uint32_t idesc_o = umma_idesc_f16(kMmaBF16, 128, D, false, true);
      const uint64_t dQ = umma_sdesc_sw128(smem_u32(sQ), 16, 1024), dK = umma_sdesc_sw128(smem_u32(sK), 16, 1024);
      const uint64_t dV = umma_sdesc_sw128(smem_u32(sV), kHalfBytes, 1024), dP = umma_sdesc_sw128(smem_u32(sP), 16, 1024);
      uint32_t kt = 0, turn = 0, done = 0;                     // tiles; items of one block; items
      Pair uses, p_of;                                         // of the query areas; steps of A and B
      for (;; ++done) {
        ok = ok && wait_item(done);
        if (!ok) break;
        const Item it = read_item(done);
        done_reading(done);
        if (it.rows == 0) break;
        const bool two = it.two(), few = it.few();
        const int N = it.steps();
        const int area = int(turn & 1u);                       // of an item of one block
        // S_x(n) = Q K^T into TMEM columns 128x .. 128x + 127.  A descriptor advances by bytes / 16.
        auto issue_s = [&](int n) -> bool {
          const int x = n & 1, a = two ? x : area;
          const uint32_t tile = kt + (two ? n >> 1 : n), st = tile % kStages;
          if ((two ? n < 2 : n == 0) && !all(mbar_wait(&bar_q[a], uses[a] & 1u))) return false;
          if (!all(mbar_wait(&bar_k_full[st], (tile / kStages) & 1u))) return false;
          tc_fence_after();
          const uint64_t da = dQ + uint32_t(a * C::kTileBytes / 16), db = dK + uint32_t(st * C::kTileBytes / 16);
  #pragma unroll
          for (int kk = 0; kk < D / 16; ++kk)
            mma_ss(lead, tmem + 128 * x, da + ((kk >> 2) * kHalfBytes + (kk & 3) * 32) / 16,
                   db + ((kk >> 2) * kHalfBytes + (kk & 3) * 32) / 16, idesc_s, kk > 0);
          commit(lead, &bar_s_full[x]);
          if (!two || x == 1) commit(lead, &bar_k_empty[st]);
          if (two ? n + 2 >= N : n + 1 == N) commit(lead, &bar_q_empty[a]);
          return true;
        };
        // O_x += P_x V, P_x in the first 64 columns of the scores, or of few rows in shared memory.
        auto issue_pv = [&](int n) -> bool {
          const int x = n & 1;
          const uint32_t tile = kt + (two ? n >> 1 : n), st = tile % kStages;
          if (!all(mbar_wait(&bar_v_seen[st], (tile / kStages) & 1u))) return false;
          if (n == 0 && done > 0 && !all(mbar_wait(&bar_o_free, (done - 1) & 1u))) return false;
          if (!all(mbar_wait(&bar_p_full[x], p_of[x] & 1u))) return false;
          p_of.up(x);
          tc_fence_after();
          const uint64_t b = dV + uint32_t(st * C::kTileBytes / 16);
          if (few) {
            const uint64_t a = dP + uint32_t(x * C::kWeights / 16);
  #pragma unroll
            for (int kk = 0; kk < kTile / 16; ++kk)
              mma_ss(lead, tmem + 256 + 128 * x, a + ((kk >> 2) * C::kWeightHalf + (kk & 3) * 32) / 16, b + kk * 2048 / 16, idesc_o,
                     n >= 2 || kk > 0);
          } else {
  #pragma unroll
            for (int kk = 0; kk < kTile / 16; ++kk)
              mma_ts(lead, tmem + 256 + 128 * x, tmem + 128 * x + kk * 8, b + kk * 2048 / 16, idesc_o, n >= 2 || kk > 0);
          }
          commit(lead, &bar_pv_done[x]);
          if (!two || x == 1) commit(lead, &bar_v_empty[st]);
          return true;
        };
        ok = issue_s(0) && (N < 2 || issue_s(1));
        for (int n = 0; ok && n < N; ++n) ok = issue_pv(n) && (n + 2 >= N || issue_s(n + 2));
        if (!ok) break;
        kt += it.t1 - it.t0;
        if (two) {
          uses.up(0);
          uses.up(1);
        } else {
          uses.up(area);
          ++turn;
        }
      }
      if (!ok && lane == 0) set_error(p.pc.err, PKV_DEVERR_TIMEOUT);
      commit(lead, &bar_drain);                                // no product may be under way when the CTA leaves
      (void)mbar_wait(&bar_drain, 0);
    } else {
      // ---------------- queries of items of one block ----------------
      const int tid = threadIdx.x - 26 * 32;
      uint32_t turn = 0;
      Pair uses;
      for (uint32_t i = 0;; ++i) {
        ok = ok && wait_item(i);
        if (!ok) break;
        const Item it = read_item(i);
        done_reading(i);
        if (it.rows == 0) break;
        if (it.two()) {
          // Not ours to fill, but to wait for: a later wait could take an earlier phase that was
          // skipped for its own.  The arrival keeps the areas' next phases from passing before that.
          for (int a = 0; a < 2 && ok; ++a) {
            ok = all(uses[a] == 0 || mbar_wait(&bar_q_empty[a], (uses[a] - 1) & 1u));
            uses.up(a);
            if (ok && lane == 0) mbar_arrive(&bar_q[a]);
          }
          if (!ok) break;
          continue;
        }
        const int a = int(turn++ & 1u);
        float* fac = factor[a][uses[a] & 1u];
        ok = load_queries<kBF16, !kWide, D, 64, 4>(smem_u32(sQ) + a * C::kTileBytes, p.q, it.q0, p.num_heads, it.h, p.group, it.f0, it.rows,
                                           it.few() ? kTile / kFewRows : 1, p.scale_log2, !kWide && p.k_scale ? __ldg(p.k_scale + it.h) : 1.f, tid,
                                           [&] { return all(uses[a] == 0 || mbar_wait(&bar_q_empty[a], (uses[a] - 1) & 1u)); },
                                           [](int) { return 0.f; }, [&](int row, float c, float) { fac[row] = c; });
        if (!ok) break;
        uses.up(a);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {                                       // (for the chain's warps too)
          for (int u = 0; u < 3; ++u) mbar_arrive(&bar_q[a]);
        }
      }
      if (!ok && lane == 0) set_error(p.pc.err, PKV_DEVERR_TIMEOUT);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 25) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

// Merges the parts of items that several CTAs worked on.  A CTA begins at most one such item, as its last;
// the other parts are the first ones of the CTAs after it.  blockIdx.x: the CTA that began it; kMergeRows
// rows each, a warp per row.
constexpr int kMergeRows = 16;
template <bool kBF16, int D>
__global__ void __launch_bounds__(kMergeThreads) chunk_merge_kernel(const ChunkParams p, int ctas, bool scaled) {
  __shared__ int slots[2 * 1024];
  __shared__ int count;
  griddep_launch_dependents();
  griddep_wait();
  const Part* headers = reinterpret_cast<const Part*>(p.parts);
  const Part a = headers[2 * blockIdx.x], b = headers[2 * blockIdx.x + 1];
  const bool second = b.rows != 0;                           // (an unfinished item behind another is the last)
  const Part me = second ? b : a;
  const int row0 = blockIdx.y * kMergeRows;
  if (me.rows == 0 || me.t0 != 0 || row0 >= me.rows) return;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, G = int(p.group.d);
  if (warp == 0) {                                           // the parts, in the order of their keys
    if (lane == 0) slots[0] = 2 * blockIdx.x + second;
    int n = 1;
    bool more = me.t1 < me.tiles;
    for (int w0 = blockIdx.x + 1; more && w0 < ctas; w0 += 32) {
      Part part = {};
      if (w0 + lane < ctas) part = headers[2 * (w0 + lane)];
      const bool same = part.rows != 0 && part.t0 != 0 && part.seq == me.seq && part.h == me.h && part.f0 == me.f0;
      const unsigned m = __ballot_sync(0xffffffffu, same);
      if (same) slots[n + __popc(m & ((1u << lane) - 1))] = 2 * (w0 + lane);
      n += __popc(m);
      more = !__any_sync(0xffffffffu, same && part.t1 >= part.tiles);
    }
    if (lane == 0) count = n;
  }
  __syncthreads();
  const int n = count;
  const uint8_t* bodies = p.parts + size_t(ctas) * 2 * sizeof(Part);
  const size_t stride = part_bytes(p.part_rows, D);
  constexpr int kVec = D / 64, kAhead = 4;                   // float2 of a lane; parts in flight
  const float vs = scaled && p.v_scale ? p.v_scale[me.h] : 1.f;
  for (int r = row0 + warp; r < min(me.rows, row0 + kMergeRows); r += kMergeThreads / 32) {
    float m = -INFINITY;
    for (int k = lane; k < n; k += 32) m = fmaxf(m, reinterpret_cast<const float2*>(bodies + slots[k] * stride)[r].x);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    float l = 0.f;
    float2 o[kVec];
#pragma unroll
    for (int c = 0; c < kVec; ++c) o[c] = make_float2(0.f, 0.f);
    for (int k0 = 0; k0 < n; k0 += kAhead) {
      float2 ml[kAhead], v[kAhead][kVec];
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        const uint8_t* body = bodies + slots[min(k0 + u, n - 1)] * stride;
        ml[u] = reinterpret_cast<const float2*>(body)[r];
        const float2* src = reinterpret_cast<const float2*>(body + part_head(p.part_rows)) + size_t(r) * (D / 2) + lane;
#pragma unroll
        for (int c = 0; c < kVec; ++c) v[u][c] = src[32 * c];
      }
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        // A part without keys for the row: its O is 0 or was never written.
        if (k0 + u >= n || ml[u].x == -INFINITY) continue;
        const float w = fast_exp2(ml[u].x - m);
        l += ml[u].y * w;
#pragma unroll
        for (int c = 0; c < kVec; ++c) {
          o[c].x += v[u][c].x * w;
          o[c].y += v[u][c].y * w;
        }
      }
    }
    const int f = me.f0 + r, row = int(p.group.quotient(f));
    const int64_t unit = (int64_t(me.q0) + row) * p.num_heads + int64_t(me.h) * G + (f - row * G);
    const float inv = l == 0.f ? 0.f : vs / l;
#pragma unroll
    for (int c = 0; c < kVec; ++c)
      reinterpret_cast<uint32_t*>(p.out)[unit * (D / 2) + 32 * c + lane] = pack2<kBF16>(o[c].x * inv, o[c].y * inv);
    if (p.lse && lane == 0) p.lse[unit] = (m + log2f(l)) * 0.6931471805599453f;
  }
}

int part_rows_of(int total_q, int num_heads, int num_kv_heads) {
  return int(std::min<int64_t>(kItemRows, int64_t(total_q) * (num_heads / num_kv_heads)));
}

template <int KV, bool kBF16, int D>
pkv_status launch(const CUtensorMap& tk, const CUtensorMap& tv, const ChunkParams& prm, cudaStream_t stream) {
  constexpr int smem = Cfg<KV, D>::kSmem;
  auto kern = chunk_kernel<KV, kBF16, D>;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess) return PKV_ERR_CUDA;
  const int ctas = num_sms();
  if (ctas < 1 || ctas > 1024) return PKV_ERR_UNSUPPORTED;   // (the merge's list)
  if (launch_pdl(kern, dim3(ctas), dim3(kThreads), smem, stream, tk, tv, prm) != cudaSuccess) return PKV_ERR_CUDA;
  return launch_pdl(chunk_merge_kernel<kBF16, D>, dim3(ctas, (prm.part_rows + kMergeRows - 1) / kMergeRows), dim3(kMergeThreads), 0, stream, prm,
                    ctas, KV != PKV_F16 && KV != PKV_BF16) == cudaSuccess
             ? PKV_OK
             : PKV_ERR_CUDA;
}

}  // namespace
}  // namespace pkv

extern "C" size_t pkv_chunk_workspace_bytes(int total_q, int num_heads, int num_kv_heads, int head_dim) {
  using namespace pkv;
  if (total_q <= 0 || num_heads <= 0 || num_kv_heads <= 0 || head_dim <= 0 || num_heads % num_kv_heads) return 0;
  return size_t(std::max(1, num_sms())) * 2 * (sizeof(Part) + part_bytes(part_rows_of(total_q, num_heads, num_kv_heads), head_dim));
}

extern "C" pkv_status pkv_paged_chunk_attention(void* out, float* lse, const void* q, pkv_dtype q_dtype,
                                                const int32_t* cu_q_lens, const int32_t* q_start_pos, int num_chunks,
                                                int total_q, int num_heads, const void* k_cache, const void* v_cache,
                                                const pkv_cache_desc* cache, const int32_t* block_tables,
                                                int max_blocks_per_seq, float scale, void* workspace,
                                                size_t workspace_bytes, pkv_stream_t stream) {
  using namespace pkv;
  pkv_status st = check_cache_desc(cache);
  if (st != PKV_OK) return st;
  if (num_chunks < 0 || total_q < 0 || num_heads <= 0 || max_blocks_per_seq < 0 || num_heads % cache->num_kv_heads)
    return PKV_ERR_INVALID_ARG;
  if (q_dtype != PKV_F16 && q_dtype != PKV_BF16) return PKV_ERR_INVALID_ARG;
  if (!(scale > 0.f) || scale > kMostScale) return PKV_ERR_INVALID_ARG;
  if ((cache->kv_dtype == PKV_F16 || cache->kv_dtype == PKV_BF16) && cache->kv_dtype != q_dtype)
    return PKV_ERR_UNSUPPORTED;
  if (cache->head_dim != 64 && cache->head_dim != 128) return PKV_ERR_UNSUPPORTED;
  if (cache->block_size != 16 && cache->block_size != 32) return PKV_ERR_UNSUPPORTED;
  if (!chunk_work_fits(num_chunks, total_q, num_heads, max_blocks_per_seq, cache)) return PKV_ERR_UNSUPPORTED;
  if (num_chunks == 0 || total_q == 0) return PKV_OK;
  if (!out || !q || !cu_q_lens || !q_start_pos || !k_cache || !v_cache || !block_tables || max_blocks_per_seq == 0)
    return PKV_ERR_INVALID_ARG;
  if (!aligned16(out) || !aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache) ||
      (reinterpret_cast<uintptr_t>(lse) & 3u) || (reinterpret_cast<uintptr_t>(cu_q_lens) & 3u) ||
      (reinterpret_cast<uintptr_t>(q_start_pos) & 3u) || (reinterpret_cast<uintptr_t>(block_tables) & 3u))
    return PKV_ERR_INVALID_ARG;
  if (!workspace || !aligned16(workspace) ||
      workspace_bytes < pkv_chunk_workspace_bytes(total_q, num_heads, cache->num_kv_heads, cache->head_dim))
    return PKV_ERR_WORKSPACE;
  if (!on_current_device(q) || !on_current_device(k_cache) || !on_current_device(v_cache) || !on_current_device(out))
    return PKV_ERR_INVALID_ARG;
  unsigned* err = error_word_ptr();
  if (!err) return PKV_ERR_CUDA;
  ChunkParams prm = {.group = Divisor(num_heads / cache->num_kv_heads)};
  prm.out = static_cast<uint8_t*>(out);
  prm.lse = lse;
  prm.q = static_cast<const uint8_t*>(q);
  prm.cu_q = cu_q_lens;
  prm.start = q_start_pos;
  prm.k_cache = static_cast<const uint8_t*>(k_cache);
  prm.v_cache = static_cast<const uint8_t*>(v_cache);
  prm.k_scale = cache->k_scale;
  prm.v_scale = cache->v_scale;
  prm.parts = static_cast<uint8_t*>(workspace);
  prm.part_rows = part_rows_of(total_q, num_heads, cache->num_kv_heads);
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
  const bool wide = cache->kv_dtype == PKV_F16 || cache->kv_dtype == PKV_BF16;
  CUtensorMap tk = {}, tv = {};
  if (wide) {                                                // boxes of 64 elements by 16 of the pool's rows
    const int64_t rows = int64_t(cache->num_blocks) * cache->num_kv_heads * cache->block_size;
    if (rows >= (int64_t(1) << 31) - 1) return PKV_ERR_UNSUPPORTED;
    auto encode = [&](CUtensorMap* m, const void* base) {
      return encode_tmap_2d(m, CU_TENSOR_MAP_DATA_TYPE_UINT16, base, uint64_t(cache->head_dim), uint64_t(rows),
                            uint64_t(cache->head_dim) * 2, 64, 16, CU_TENSOR_MAP_SWIZZLE_128B);
    };
    if (!encode(&tk, k_cache) || !encode(&tv, v_cache)) return PKV_ERR_CUDA;
  }
  const bool d128 = cache->head_dim == 128, bf = q_dtype == PKV_BF16;
  switch (cache->kv_dtype) {
    case PKV_F16: return d128 ? launch<PKV_F16, false, 128>(tk, tv, prm, s) : launch<PKV_F16, false, 64>(tk, tv, prm, s);
    case PKV_BF16: return d128 ? launch<PKV_BF16, true, 128>(tk, tv, prm, s) : launch<PKV_BF16, true, 64>(tk, tv, prm, s);
    case PKV_FP8_E4M3:
      return bf ? (d128 ? launch<PKV_FP8_E4M3, true, 128>(tk, tv, prm, s) : launch<PKV_FP8_E4M3, true, 64>(tk, tv, prm, s))
                : (d128 ? launch<PKV_FP8_E4M3, false, 128>(tk, tv, prm, s) : launch<PKV_FP8_E4M3, false, 64>(tk, tv, prm, s));
    default:
      return bf ? (d128 ? launch<PKV_FP4_E2M1, true, 128>(tk, tv, prm, s) : launch<PKV_FP4_E2M1, true, 64>(tk, tv, prm, s))
                : (d128 ? launch<PKV_FP4_E2M1, false, 128>(tk, tv, prm, s) : launch<PKV_FP4_E2M1, false, 64>(tk, tv, prm, s));
  }
}
