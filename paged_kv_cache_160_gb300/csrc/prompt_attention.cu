// prompt_attention: causal attention of packed prompts over keys and values given as plain rows.
//
// Mathematics: row r of a sequence with Lq query and Lk key rows attends keys 0 .. r + Lk - Lq.  One
// pass over the keys in tiles of 128 with the running maximum m and sum l of the softmax (in units
// of log2): P = 2^(s c - m), O = O 2^(m_old - m) + P V, out = O / l.
//
// GB300 design: a CTA holds two row blocks of 128 rows that read the same keys, so every K/V tile feeds 256
// rows: query rows of one head, or of all query heads of a kv head (Blocks).  S = Q K^T and O += P V run on
// tcgen05 with S, P and O in tensor memory; Q, K and V arrive by TMA straight from the packed rows (any row
// stride).  P is rounded to the type of V, as both operands of a product share a type (2^-8 of each weight in
// bf16, 2^-11 in f16); l sums the unrounded fp32 values.
//
// Bound: the tensor cores, and the exponentials beside them (a 128 x 128 tile is 16,384 of them, about as
// many cycles of the special function units as of its two products).  Measured in a graph: 8192 tokens,
// 32 heads over 8, D 128: 322 us, 1.71 PFLOP/s of causal pairs; 16 prompts of 64 to 2048 tokens, 28 heads
// over 4: 208 us; 512 rows behind 3584 keys: 33 us.  The products alone, without a softmax, take 297 us of
// the first.
#include <algorithm>
#include <type_traits>

#include "pkv_device.cuh"
#include "pkv_host.h"
#include "umma_issue.cuh"

namespace pkv {
namespace {

constexpr int kTile = 128;                    // query rows of a block, keys of a tile
constexpr int kThreads = 640;
constexpr uint32_t kTmemCols = 512;           // S_A | S_B | O_A | O_B, 128 columns each
constexpr int kHalfBytes = kTile * 128;       // [128 rows][64 elements] of 2 bytes
constexpr float kRescaleThreshold = 8.f;      // log2 units

struct PromptParams {
  uint8_t* out;
  const int32_t* cu_q;
  const int32_t* cu_k;
  int64_t out_stride;     // elements
  const uint8_t* v;
  int64_t v_stride;       // elements
  int num_seqs;
  int compact;            // items are numbered sequence by sequence (see item_of)
  int total_q;
  int total_k;
  int max_q_len;
  int num_heads;
  int num_kv_heads;
  float scale_log2;
  unsigned* err;
  Divisor group;          // query heads per kv head
};

// Asks for a CTA of the grid that has not started: the hardware cancels its launch and writes its index
// (or that there is none) to 16 bytes at `response`, completing 16 bytes on `bar`.
__device__ __forceinline__ void ask_for_cta(void* response, uint64_t* bar) {
  asm volatile("clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];" ::"r"(
                   smem_u32(response)),
               "r"(smem_u32(bar))
               : "memory");
}
// The answer: whether there was one, and its block index.
__device__ __forceinline__ bool read_cta(const void* response, int& x, int& y, int& z) {
  uint32_t got, a, b, c;
  asm volatile(
      "{\n\t.reg .b128 r;\n\t.reg .pred p;\n\t"
      "mov.u32 %0, 0;\n\tmov.u32 %1, 0;\n\tmov.u32 %2, 0;\n\t"
      "ld.shared.b128 r, [%4];\n\t"
      "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, r;\n\t"
      "selp.u32 %3, 1, 0, p;\n\t"
      "@p clusterlaunchcontrol.query_cancel.get_first_ctaid.v4.b32.b128 {%0, %1, %2, _}, r;\n\t}\n"
      : "=&r"(a), "=&r"(b), "=&r"(c), "=&r"(got)
      : "r"(smem_u32(response))
      : "memory");
  x = int(a);
  y = int(b);
  z = int(c);
  return got != 0;
}

// ---------------------------------------------------------------------------------------
// A CTA works on items: two row blocks A and B of 128 query rows that read the same keys.  The grid
// has a CTA for every possible item; the ones that the GPU can hold take over the items of those that
// have not started (ask_for_cta), so that barriers and TMEM are set up once per SM, the next item's
// loads and first products run while the last rows of this one are written, and an SM that is done
// early takes the next item.  (A CTA per item spent 7 us outside the tile loop.)
//   warps 0-7 : softmax of block A, warps 8-15: of block B; two threads per query row, one for each half
//               of the tile's keys.  A tile's way from its scores to its product with V is a chain that
//               only the other block's products cover (3200 cycles for both blocks, about 2400 of them
//               products), so the softmax is spread over twice the threads: one thread per row took
//               390 us for a prompt of 8192 tokens where two take 381.
//   warp 16   : TMA producer of Q, K and V; asks for the next item and hands it to the other warps through
//               shared memory (16 packed prompts took 226 us when every warp read the lengths by itself, 218
//               since, and small items gain most: 4 us each instead of 7)
//   warp 17   : TMEM owner and MMA issuer, in the order S_A(0) S_B(0) | PV_A(t) S_A(t+1) PV_B(t) S_B(t+1) | ...
//               so that one block's softmax overlaps the other's products
//   warps 18-19: pass every V tile on to warp 17, having looked at those that some rows see only in part (from
//               Item::masked on): 0 * V must not turn the rows' other keys into NaN.  V rows past the sequence's
//               end become zeros, and so do non-finite values, which the rows that do see them get back at the end.
// Every barrier's phases are counted over all items by each of its users.
// ---------------------------------------------------------------------------------------
template <int D>
struct Cfg {
  static constexpr int kTileBytes = D / 64 * kHalfBytes;          // 128 rows of Q, K or V
  static constexpr int kStages = D == 128 ? 2 : 4;                // K and V tiles in flight
  static constexpr int kStageRows = 8;                            // half rows of output that a warp stages at a time
  static constexpr int kOutBytes = kStageRows * D;                // (16-bit half rows)
  static constexpr int kSmem = (2 + 2 * kStages) * kTileBytes + 16 * kOutBytes;
};

struct Item {
  int h;                  // kv head
  int q0, k0, Lq, Lk;     // the sequence's first rows and lengths
  int rows;               // query rows to compute (at most max_q_len)
  int e0;                 // block A is row block e0 of the (sequence, kv head), B the next one
  int t0;                 // first key tile
  int masked;             // key tiles from here on are seen only in part by some rows (tile index of the sequence)
  int na, nb, n;          // key tiles that A and B walk from there, and the larger
  bool live;              // there are such rows
};

// What a row block holds: 128 rows of one query head; or, packed, `rows` rows of all G query heads of a kv head,
// block row i being row i / G of head i mod G.  Blocks are numbered query tile by query tile, its heads inside.
struct Blocks {
  int rows;               // query rows of a block
  int per_tile;           // blocks of the same rows
  __host__ __device__ Blocks(bool packed, int G) : rows(packed ? kTile / G : kTile), per_tile(packed ? 1 : G) {}
  __device__ __forceinline__ int first_row(int e) const { return e / per_tile * rows; }
};

// A sequence: its rows, or none of them where the lengths are inconsistent.
struct Seq {
  int q0, k0, Lq, Lk, rows;
  bool bad;
  __device__ __forceinline__ Seq(const PromptParams& p, int s) {
    q0 = p.cu_q[s];
    k0 = p.cu_k[s];
    Lq = p.cu_q[s + 1] - q0;
    Lk = p.cu_k[s + 1] - k0;
    bad = q0 < 0 || k0 < 0 || Lq < 0 || Lk < 0 || Lq > p.total_q - q0 || Lk > p.total_k - k0;
    rows = bad ? 0 : min(Lq, p.max_q_len);
  }
  // Items of one of its kv heads: two row blocks each.
  __device__ __forceinline__ int items(const Blocks& b) const { return ((rows + b.rows - 1) / b.rows * b.per_tile + 1) / 2; }
};

// The item of a sequence's kv head h with row blocks 2 * level and 2 * level + 1.
__device__ __forceinline__ Item item_at(const PromptParams& p, const Blocks& blocks, int h, int s, int level) {
  const Seq q(p, s);
  Item it;
  it.h = h;
  it.q0 = q.q0;
  it.k0 = q.k0;
  it.Lq = q.Lq;
  it.Lk = q.Lk;
  it.rows = q.rows;
  it.e0 = 2 * level;
  it.live = unsigned(level) < unsigned(q.items(blocks));
  // Key tiles that the rows of block e attend (0: none, or no such rows).
  auto tiles_of = [&](int e) -> int {
    const int r0 = blocks.first_row(e);
    if (r0 >= it.rows) return 0;
    const int keys = min(it.Lq, r0 + blocks.rows) + it.Lk - it.Lq;
    return keys > 0 ? (keys + kTile - 1) / kTile : 0;
  };
  it.na = it.live ? tiles_of(it.e0) : 0;
  it.nb = it.live ? tiles_of(it.e0 + 1) : 0;
  it.n = max(it.na, it.nb);
  it.t0 = 0;
  it.masked = max(0, blocks.first_row(it.e0) + it.Lk - it.Lq + 1) / kTile;   // the earlier block's first row decides
  return it;
}

// Adds to v the non-finite values among V[j][d .. d + 31], d counting the elements of the packed row, of keys
// j0 .. j1 - 1.
template <bool kBF16>
__device__ __forceinline__ void add_non_finite(const PromptParams& p, int k0, int j0, int j1, int d, float (&v)[32]) {
  for (int j = j0; j < j1; ++j) {
    const uint4* row = reinterpret_cast<const uint4*>(p.v + ((int64_t(k0) + j) * p.v_stride + d) * 2);
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const uint4 u = row[c];
      const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float2 f = unpack2<kBF16>(w[k]);
        if (!(fabsf(f.x) < INFINITY)) v[8 * c + 2 * k] += f.x;
        if (!(fabsf(f.y) < INFINITY)) v[8 * c + 2 * k + 1] += f.y;
      }
    }
  }
}

constexpr int kMaxSeqs = 65535;
constexpr int kItems = 4;                                    // items on their way from the producer to the other warps
constexpr int kSeqChunk = 32;                                // sequences per entry of the compact numbering's table

// The item of block index (x, y, z), for a whole warp.
//   Level by level (compact 0): x is the kv head, y the sequence, z counts the levels of the longest
// sequence down.  The hardware starts CTAs with x fastest and z slowest: the items that walk the most
// keys come first.  Shorter sequences' indexes have nothing to do.
//   Sequence by sequence (compact 1), where those would be too many: x counts kv heads, then a sequence's
// levels down, then sequences; `first` holds the number of every kSeqChunk-th sequence's first item.
__device__ __forceinline__ Item item_of(const PromptParams& p, const Blocks& blocks, int x, int y, int z, int nz,
                                        const int* first, int lane) {
  if (!p.compact) return item_at(p, blocks, x, y, nz - 1 - z);
  const int h = x % p.num_kv_heads, j = x / p.num_kv_heads;
  int lo = 0, hi = (p.num_seqs + kSeqChunk - 1) / kSeqChunk; // the chunk of item j: first[lo] <= j < first[hi]
  if (j >= first[hi]) return Item{};
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (first[mid] <= j) lo = mid; else hi = mid;
  }
  const int s = lo * kSeqChunk + lane, mine = s < p.num_seqs ? Seq(p, s).items(blocks) : 0;
  int sum = mine;                                            // inclusive scan over the chunk
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, sum, o);
    if (lane >= o) sum += v;
  }
  const int rest = j - first[lo];
  const unsigned past = __ballot_sync(0xffffffffu, sum > rest);
  if (past == 0) return Item{};                              // (lengths that contradict one another)
  const int l = __ffs(past) - 1;
  const int before = __shfl_sync(0xffffffffu, sum - mine, l), count = __shfl_sync(0xffffffffu, mine, l);
  return item_at(p, blocks, h, lo * kSeqChunk + l, count - 1 - (rest - before));
}

// Part `part` of `parts` of an item's key tiles.
__device__ __forceinline__ void take_part(Item& it, int part, int parts) {
  const int t1 = int(int64_t(it.n) * (part + 1) / parts);
  it.t0 = int(int64_t(it.n) * part / parts);
  it.na = max(0, min(it.na, t1) - it.t0);
  it.nb = max(0, min(it.nb, t1) - it.t0);
  it.n = max(it.na, it.nb);
}

// The shared::cluster address of this CTA's shared address `addr` in the CTA of the given rank.
__device__ __forceinline__ uint32_t cluster_addr(uint32_t addr, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
// Copies `bytes` (a multiple of 16) from this CTA's shared memory to another CTA's of the cluster,
// completing on that CTA's mbarrier; dst and bar are shared::cluster addresses.
__device__ __forceinline__ void copy_to_cta(uint32_t dst, uint32_t src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.shared::cta.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "r"(src), "r"(bytes), "r"(bar)
               : "memory");
}

// kSplit: a cluster of 2 or 4 CTAs works on one item, each on a part of the key tiles (taken when there
// are fewer items than SMs; see launch).  Each CTA finishes an equal share of the rows: one of the two
// blocks, or 64 rows of one.  The others send it those rows, unnormalised, with their maxima and sums, by
// bulk copies from their idle K/V stages to its idle Q area (and the place of its own rows).  Reading
// them from the other CTA's shared memory with loads took 14 us instead.
template <bool kBF16, int D, bool kSplit, bool kPacked>
__global__ void __launch_bounds__(kThreads, 1)
    prompt_kernel(const __grid_constant__ CUtensorMap tmq, const __grid_constant__ CUtensorMap tmk,
                  const __grid_constant__ CUtensorMap tmv, const PromptParams p) {
  using C = Cfg<D>;
  constexpr int kStages = C::kStages;
  extern __shared__ __align__(1024) uint8_t smem[];
  __shared__ __align__(16) uint4 response;                   // ask_for_cta's answer
  __shared__ __align__(8) uint64_t bar_answer;               // it has come
  __shared__ __align__(16) int4 items[kItems][3];            // the items, by number mod kItems (see read_item)
  __shared__ __align__(8) uint64_t bar_item[kItems], bar_item_read[kItems];   // one is there / the warps have read it
  // Q_x landed / no product reads it any more; K, V tiles likewise; S_x ready; P_x ready; PV_x done; O_x read.
  __shared__ __align__(8) uint64_t bar_q[2], bar_q_empty[2], bar_k_full[kStages], bar_k_empty[kStages], bar_v_full[kStages],
      bar_v_empty[kStages], bar_s_full[2], bar_p_full[2], bar_pv_done[2], bar_o_free[2],
      bar_v_seen[kStages];                                   // V landed and, from tile `masked` on, was looked at
  __shared__ uint32_t tmem_base_sh;
  __shared__ float exchange[2][2][2][kTile];                 // [block][step parity][key half][row]
  __shared__ int first_item[kSplit ? 1 : (kMaxSeqs + kSeqChunk - 1) / kSeqChunk + 1];
  __shared__ int masked_item[2 * kItems];                    // by item number modulo that: the last such item that
                                                             // non-finite values were taken out for, + 1
  __shared__ __align__(16) float2 part_ml[2][kSplit ? kTile : 1];   // [block][row]: maximum and sum over this CTA's keys
  __shared__ __align__(16) float2 recv_ml[3][kSplit ? kTile : 1];   // [sender][row of this CTA's share]
  __shared__ __align__(8) uint64_t bar_recv;
  __shared__ uint32_t fine[2][2][2][4];                      // [block][step parity][key half][row quarter]: the warp goes on
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;   // uniform in the warp

  if (smem_u32(smem) & 1023u) {                              // the 128-byte swizzle needs 1 KB alignment
    if (threadIdx.x == 0) set_error(p.err, PKV_DEVERR_CHUNK);
    return;
  }
  uint8_t* sQ = smem;                                        // [block][64-dim half][128 rows]
  uint8_t* sK = smem + 2 * C::kTileBytes;                    // [stage][64-dim half][128 rows]
  uint8_t* sV = sK + kStages * C::kTileBytes;
  uint8_t* sOut = sV + kStages * C::kTileBytes;              // [softmax warp][kStageRows][half a row]
  if (threadIdx.x == 0) {
    prefetch_tensormap(&tmq);
    prefetch_tensormap(&tmk);
    prefetch_tensormap(&tmv);
    mbar_init(&bar_recv, 1);
    mbar_init(&bar_answer, 1);
    for (int i = 0; i < 2 * kItems; ++i) masked_item[i] = 0;
    for (int i = 0; i < kItems; ++i) {
      mbar_init(&bar_item[i], 1);
      mbar_init(&bar_item_read[i], kThreads / 32 - 1);       // every warp but the producer
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bar_q[i], 1);
      mbar_init(&bar_q_empty[i], 1);
      mbar_init(&bar_s_full[i], 1);
      mbar_init(&bar_p_full[i], 8);                          // one arrival per softmax warp
      mbar_init(&bar_pv_done[i], 1);
      mbar_init(&bar_o_free[i], 8);
    }
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&bar_k_full[i], 1);
      mbar_init(&bar_k_empty[i], 1);
      mbar_init(&bar_v_full[i], 1);
      mbar_init(&bar_v_empty[i], 1);
      mbar_init(&bar_v_seen[i], 2);
    }
    fence_mbar_init();
  }
  if (warp == 17) {
    tmem_alloc(&tmem_base_sh, kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_base_sh;

  // Only the set-up above may run before the previous kernel on the stream has finished.
  griddep_wait();
  const int G = int(p.group.d);
  const Blocks blocks(kPacked, G);
  auto all = [](bool v) -> bool { return __all_sync(0xffffffffu, v); };
  // Item number i, once its barrier's phase is complete; na = -1: there is none.
  auto read_item = [&](uint32_t i) -> Item {
    const int4 a = items[i % kItems][0], b = items[i % kItems][1], c = items[i % kItems][2];
    Item it;
    it.h = a.x;
    it.q0 = a.y;
    it.k0 = a.z;
    it.Lq = a.w;
    it.Lk = b.x;
    it.rows = b.y;
    it.e0 = b.z;
    it.t0 = b.w;
    it.masked = c.x;
    it.na = c.y;
    it.nb = c.z;
    it.n = max(it.na, it.nb);
    it.live = c.w != 0;
    return it;
  };
  // The same for a warp that works on it; the slot may be used again.
  auto take_item = [&](uint32_t i) -> Item {
    const Item it = read_item(i);
    __syncwarp();
    if (lane == 0) mbar_arrive(&bar_item_read[i % kItems]);
    return it;
  };
  auto wait_item = [&](uint32_t i) -> bool { return all(mbar_wait(&bar_item[i % kItems], i / kItems & 1u)); };
  // Block e's rows that exist, and the query row of block row r.
  auto rows_of = [&](const Item& it, int e) -> int {
    const int rows = it.rows - blocks.first_row(e);
    return kPacked ? min(rows, blocks.rows) * G : min(rows, kTile);
  };
  auto query_row = [&](int e, int r) -> int { return blocks.first_row(e) + (kPacked ? int(p.group.quotient(r)) : r); };
  // Writes a warp's 32 half rows of block e, one per lane as 16-bit pairs: kStageRows at a time through
  // the warp's own staging area (16-byte chunk c of row rr at c ^ rr against bank conflicts), so that the
  // warp writes whole runs.  (Straight from the registers a store touches 32 lines; 16 packed prompts took
  // 227 us that way, 218 with this.)
  auto write_rows = [&](const Item& it, int e, int hf, int quarter, uint8_t* area, const uint32_t (&o)[D / 4]) {
    int left = rows_of(it, e) - 32 * quarter;                // of the block's rows, from the warp's first on
    if (left <= 0) return;
    constexpr int kChunks = D / 16, kRowBytes = D, kRowsPerStore = 32 / kChunks;   // of half rows
    static_assert(kRowsPerStore <= C::kStageRows && kChunks * 16 == kRowBytes, "whole stores of a staged part");
    const uint32_t stage = smem_u32(area);
    const int rr = lane % C::kStageRows, rsub = lane / kChunks, chunk = lane % kChunks;
    const uint32_t put = stage + rr * kRowBytes, turn = rr & (kChunks - 1);
    const int64_t step = p.out_stride * (2 * kRowsPerStore);
    uint8_t* dst = p.out + 16 * chunk +
                   ((int64_t(it.q0) + blocks.first_row(e)) * p.out_stride + int64_t(it.h * G) * D + D / 2 * hf) * 2;
    if (!kPacked) dst += ((32 * quarter + rsub) * p.out_stride + int64_t(e % G) * D) * 2;
    left -= rsub;
#pragma unroll
    for (int k = 0; k < 32 / C::kStageRows; ++k) {
      if (lane / C::kStageRows == k) {
#pragma unroll
        for (int c = 0; c < kChunks; ++c) sts128(put + ((c ^ turn) << 4), o[4 * c], o[4 * c + 1], o[4 * c + 2], o[4 * c + 3]);
      }
      __syncwarp();
#pragma unroll
      for (int u = 0; u < C::kStageRows / kRowsPerStore; ++u) {
        const int from = u * kRowsPerStore + rsub;
        const uint4 v = lds128(stage + from * kRowBytes + ((chunk ^ (from & (kChunks - 1))) << 4));
        if constexpr (kPacked) {
          const int i = 32 * quarter + k * C::kStageRows + from, row = int(p.group.quotient(i));
          if (left > 0) *reinterpret_cast<uint4*>(dst + (row * p.out_stride + int64_t(i - row * G) * D) * 2) = v;
        } else {
          if (left > 0) *reinterpret_cast<uint4*>(dst) = v;
          dst += step;
        }
        left -= kRowsPerStore;
      }
      __syncwarp();
    }
  };
  // What a row gets back of element c of its half row in place of the non-finite values taken out of V.
  auto give_back = [&](const Item& it, int row, int hf, int c, float (&v)[32]) {
    add_non_finite<kBF16>(p, it.k0, max(it.masked, it.t0) * kTile,
                          min(min(row + it.Lk - it.Lq + 1, it.Lk), (it.t0 + it.n) * kTile),
                          it.h * D + D / 2 * hf + c, v);
  };
  int bx = blockIdx.x, by = blockIdx.y, bz = blockIdx.z;
  int part = 0, parts = 1;
  if constexpr (kSplit) {
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(parts));
    part = int(cluster_ctarank());
    bx /= parts;
  }
  if constexpr (!kSplit) {
    if (p.compact) {                                         // the table of the sequences' first items
      const int chunks = (p.num_seqs + kSeqChunk - 1) / kSeqChunk;
      for (int c = threadIdx.x; c < chunks; c += kThreads) {
        int sum = 0;
        for (int s = c * kSeqChunk; s < min(p.num_seqs, (c + 1) * kSeqChunk); ++s) sum += Seq(p, s).items(blocks);
        first_item[c + 1] = sum;
      }
      __syncthreads();
      if (warp == 0) {
        int total = 0;
        for (int c0 = 0; c0 < chunks; c0 += 32) {
          int v = c0 + lane < chunks ? first_item[c0 + lane + 1] : 0;
#pragma unroll
          for (int o = 1; o < 32; o <<= 1) {
            const int w = __shfl_up_sync(0xffffffffu, v, o);
            if (lane >= o) v += w;
          }
          if (c0 + lane < chunks) first_item[c0 + lane + 1] = total + v;
          total += __shfl_sync(0xffffffffu, v, 31);
        }
        if (lane == 0) first_item[0] = 0;
      }
      __syncthreads();
    }
  }
  auto this_item = [&]() -> Item {
    Item it = item_of(p, blocks, bx, by, bz, gridDim.z, first_item, lane);
    if constexpr (kSplit) take_part(it, part, parts);
    return it;
  };

  // Item `it` as number i, by the producer (one lane).
  auto put_item = [&](uint32_t i, const Item& it) {
    items[i % kItems][0] = make_int4(it.h, it.q0, it.k0, it.Lq);
    items[i % kItems][1] = make_int4(it.Lk, it.rows, it.e0, it.t0);
    items[i % kItems][2] = make_int4(it.masked, it.na, it.nb, it.live);
    mbar_arrive(&bar_item[i % kItems]);
  };
  if (warp == 16) {
    const Item it = this_item();
    if (lane == 0) put_item(0, it);
  }
  const bool first = (bx | by | bz | part) == 0;             // one CTA of the grid looks the lengths over
  __syncthreads();

  if (warp < 16) {
    if constexpr (!kSplit) asm volatile("setmaxnreg.inc.sync.aligned.u32 104;");   // 512 * 104 + 128 * 64 = 640 * 96
    // ---------------- softmax: two threads per query row ----------------
    const int x = warp >> 3, hf = (warp >> 2) & 1;   // row block; half of the keys (and of O)
    const int quarter = warp & 3, r = 32 * quarter + lane;   // TMEM lane == row of the block
    const uint32_t lane_off = uint32_t(32 * quarter) << 16;
    constexpr int kKeys = kTile / 2, kODims = D / 2;
    const float slog = p.scale_log2;                         // > 0, so max(s) * slog = max(s * slog)
    const uint32_t tS = tmem + 128 * x + lane_off + kKeys * hf;   // scores, and P over them
    const uint32_t tO = tmem + 256 + 128 * x + lane_off + kODims * hf;
    // The two warps of a row quarter meet here, once per tile and once per item, also after a wait
    // gave up: then they only walk on to the item's end, so that neither is left waiting for the other.
    auto meet = [&]() { asm volatile("bar.sync %0, 64;" ::"r"(1 + 4 * x + quarter) : "memory"); };
    bool ok = true;
    uint32_t steps = 0, meets = 0;                           // this block's steps; meetings
    for (uint32_t i = 0; ok; ++i) {
      const Item it = take_item(i);
      if (it.na < 0) break;
      const int e = it.e0 + x, row = query_row(e, r), shift = it.Lk - it.Lq;
      const int nx = x == 0 ? it.na : it.nb;
      float m = -INFINITY, l = 0.f;                          // m of the row, l of this thread's keys
      for (int t = 0; t < nx; ++t, ++meets) {
        const int kb = (it.t0 + t) * kTile;
        // Waiting for PV(t - 1) on every tile keeps that barrier at most one phase ahead of this wait.
        ok = all(ok && mbar_wait(&bar_s_full[x], (steps + t) & 1u) &&
                 (t == 0 || mbar_wait(&bar_pv_done[x], (steps + t - 1) & 1u)));
        if (!ok) {
          meet();
          continue;
        }
        tc_fence_after();
        const int lim = min(row + shift + 1, it.Lk) - kb - kKeys * hf;   // keys 0 .. lim - 1 are attended
        float s[kKeys];
#pragma unroll
        for (int cc = 0; cc < kKeys / 32; ++cc) tmem_ld32(tS + 32 * cc, *reinterpret_cast<float(*)[32]>(s + 32 * cc));
        tmem_wait_ld();
        if (lim < kKeys) {
#pragma unroll
          for (int c = 0; c < kKeys; ++c) s[c] = c < lim ? s[c] : -INFINITY;
        }
        float c4[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
        for (int c = 4; c < kKeys; c += 8) {
#pragma unroll
          for (int u = 0; u < 4; ++u)
            if (c + 2 * u + 1 < kKeys) c4[u] = fmax3(c4[u], s[c + 2 * u], s[c + 2 * u + 1]);
        }
        const float mine = fmaxf(fmaxf(c4[0], c4[1]), fmaxf(c4[2], c4[3]));
        float* xm = &exchange[x][meets & 1][0][r];
        xm[kTile * hf] = mine;
        meet();
        const float mt = fmaxf(mine, xm[kTile * (hf ^ 1)]) * slog;
        const bool grow = mt > m + kRescaleThreshold;        // also true for the first tile
        const float m_prev = m;
        if (grow) m = mt;
        // P over S (keys 2e, 2e + 1 in column e).  A row without keys so far has m = -inf and every
        // s = -inf: m = 0 then gives P = 0.
        const float mu = m == -INFINITY ? 0.f : m;
        const uint64_t sl2 = pack_f32x2(slog, slog), nm2 = pack_f32x2(-mu, -mu);
        uint64_t acc0 = pack_f32x2(0.f, 0.f), acc1 = acc0;
#pragma unroll
        for (int hb = 0; hb < kKeys / 32; ++hb) {
          uint32_t w[16];
#pragma unroll
          for (int c = 0; c < 16; ++c) {
            const int c0 = 32 * hb + 2 * c;
            const uint64_t x2 = fma_f32x2(pack_f32x2(s[c0], s[c0 + 1]), sl2, nm2);
            const float pa = fast_exp2(lo_f32(x2)), pb = fast_exp2(hi_f32(x2));
            const uint64_t p2 = pack_f32x2(pa, pb);
            if (c & 1) acc1 = add_f32x2(acc1, p2);
            else acc0 = add_f32x2(acc0, p2);
            w[c] = pack2<kBF16>(pa, pb);
          }
          tmem_st16u(tS + 16 * hb, w);
        }
        if (__any_sync(0xffffffffu, grow && t >= 1)) {       // rescale this thread's half of O
          const float alpha = (grow && m_prev != -INFINITY) ? fast_exp2(m_prev - m) : 1.f;
#pragma unroll
          for (int cc = 0; cc < kODims / 32; ++cc) {
            float v[32];
            tmem_ld32(tO + 32 * cc, v);
            tmem_wait_ld();
#pragma unroll
            for (int c = 0; c < 32; ++c) v[c] *= alpha;
            tmem_st32(tO + 32 * cc, v);
          }
          if (grow) l *= alpha;
        }
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar_p_full[x]);
        const uint64_t acc = add_f32x2(acc0, acc1);
        l += lo_f32(acc) + hi_f32(acc);
      }
      steps += nx;
      // ---------------- output ----------------
      ok = all(ok && (nx == 0 || mbar_wait(&bar_pv_done[x], (steps - 1) & 1u)));
      tc_fence_after();
      if (!kSplit) ok = ok && wait_item(i + 1);              // here, so that both warps go on or none
      float* xl = &exchange[x][meets & 1][0][r];
      xl[kTile * hf] = l;
      if (lane == 0) fine[x][meets & 1][hf][quarter] = ok;
      meet();
      l += xl[kTile * (hf ^ 1)];
      ok = ok && fine[x][meets & 1][hf ^ 1][quarter] != 0;   // both warps go on, or none
      ++meets;
      if constexpr (kSplit) {                                // the rows are finished below
        // m = -inf stands for no keys; a row whose scores are all NaN has some.
        if (hf == 0) part_ml[x][r] = make_float2(m == -INFINITY && l != 0.f ? 0.f : m, l);
        break;
      }
      const bool taken = *static_cast<volatile int*>(&masked_item[i % (2 * kItems)]) == int(i) + 1;
      uint32_t o[kODims / 2];
      if (nx > 0 && ok) {
        float v[kODims];
#pragma unroll
        for (int cc = 0; cc < kODims / 32; ++cc) tmem_ld32(tO + 32 * cc, *reinterpret_cast<float(*)[32]>(v + 32 * cc));
        tmem_wait_ld();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar_o_free[x]);          // the next item may overwrite O
        if (taken) {
#pragma unroll
          for (int cc = 0; cc < kODims / 32; ++cc)
            give_back(it, row, hf, 32 * cc, *reinterpret_cast<float(*)[32]>(v + 32 * cc));
        }
        const float inv = l == 0.f ? 0.f : 1.f / l;          // l = 0: a row without keys, whose O is 0; NaN stays
        const uint64_t inv2 = pack_f32x2(inv, inv);
#pragma unroll
        for (int c = 0; c < kODims / 2; ++c) {
          const uint64_t y = mul_f32x2(pack_f32x2(v[2 * c], v[2 * c + 1]), inv2);
          o[c] = pack2<kBF16>(lo_f32(y), hi_f32(y));
        }
      } else {
#pragma unroll
        for (int c = 0; c < kODims / 2; ++c) o[c] = 0u;
      }
      if (ok) write_rows(it, e, hf, quarter, sOut + warp * C::kOutBytes, o);
    }
    if (!ok && lane == 0) set_error(p.err, PKV_DEVERR_TIMEOUT);
  } else {
    if constexpr (!kSplit) asm volatile("setmaxnreg.dec.sync.aligned.u32 64;");
    if (warp == 16) {
      // ---------------- TMA producer ----------------
      const uint64_t pol_q = l2_policy_evict_first();
      const uint64_t pol_kv = l2_policy_evict_last();          // re-read by the other heads and query tiles
      bool ok = true;
      uint32_t kt = 0, q_of[2] = {0, 0}, answers = 0;          // K/V tiles; Q blocks A, B; answers so far
      auto ask = [&]() {
        fence_proxy_async_smem();                              // the answer comes after the last one was read
        __syncwarp();
        if (lane == 0) {
          mbar_arrive_expect_tx(&bar_answer, 16);
          ask_for_cta(&response, &bar_answer);
        }
      };
      Item it = read_item(0);
      for (uint32_t i = 0;; ++i) {
        if (!kSplit) ask();                                    // for the item after this one
        // The queries of block x, once the products with the last ones are done (never called without keys).
        auto load_q = [&](int x) {
          ok = ok && all(q_of[x] == 0 || mbar_wait(&bar_q_empty[x], (q_of[x] - 1) & 1u));
          if (!ok) return;
          if (lane == 0) {
            mbar_arrive_expect_tx(&bar_q[x], kPacked ? blocks.rows * G * D * 2 : C::kTileBytes);
            const int e = it.e0 + x;
            for (int d = 0; d < D / 64; ++d)
              tma_load_3d(sQ + x * C::kTileBytes + d * kHalfBytes, &tmq, &bar_q[x], 64 * d,
                          it.h * G + (kPacked ? 0 : e % G), it.q0 + blocks.first_row(e), pol_q);
          }
          ++q_of[x];
        };
        for (int t = 0; ok && t < it.n; ++t, ++kt) {
          const uint32_t st = kt % kStages, par = (kt / kStages - 1) & 1u;
          ok = all(kt < uint32_t(kStages) || mbar_wait(&bar_k_empty[st], par));
          if (ok && lane == 0) {
            mbar_arrive_expect_tx(&bar_k_full[st], C::kTileBytes);
            for (int d = 0; d < D / 64; ++d)
              tma_load_3d(sK + st * C::kTileBytes + d * kHalfBytes, &tmk, &bar_k_full[st], 64 * d, it.h,
                          it.k0 + (it.t0 + t) * kTile, pol_kv);
          }
          const bool k_ok = ok;                                // a K tile is on its way
          if (t == 0 && it.na > 0) load_q(0);
          const bool v_ok = ok && all(kt < uint32_t(kStages) || mbar_wait(&bar_v_empty[st], par));
          ok = v_ok;
          if (!ok) {
            if (k_ok) (void)mbar_wait(&bar_k_full[st], (kt / kStages) & 1u);
            break;
          }
          if (lane == 0) {
            mbar_arrive_expect_tx(&bar_v_full[st], C::kTileBytes);
            for (int d = 0; d < D / 64; ++d)
              tma_load_3d(sV + st * C::kTileBytes + d * kHalfBytes, &tmv, &bar_v_full[st], 64 * d, it.h,
                          it.k0 + (it.t0 + t) * kTile, pol_kv);
          }
          if (t == 0 && it.nb > 0) load_q(1);
        }
        if (kSplit) break;
        // The next item, past those without rows.  Also after a wait gave up: no answer may still be on
        // its way when the CTA leaves.
        bool got = false;
        while (true) {
          const bool came = all(mbar_wait(&bar_answer, answers & 1u));
          ++answers;
          ok = ok && came;
          if (!ok) break;
          got = read_cta(&response, bx, by, bz);
          if (!got) break;
          it = this_item();
          if (it.live) break;
          ask();
        }
        ok = ok && (i + 1 < kItems || all(mbar_wait(&bar_item_read[(i + 1) % kItems], ((i + 1) / kItems - 1) & 1u)));
        if (!ok) break;
        if (!got) it.na = -1;
        if (lane == 0) put_item(i + 1, it);
        if (!got) break;
      }
      // Drain: the last loads of each stage have landed and the commits that release the stages and Q
      // have arrived before the CTA may leave (each wait bounded).
      if (!ok && lane == 0) set_error(p.err, PKV_DEVERR_TIMEOUT);
      for (int x = 0; x < 2; ++x) {
        if (q_of[x] > 0) (void)mbar_wait(&bar_q[x], (q_of[x] - 1) & 1u);
        if (ok && q_of[x] > 0) ok = mbar_wait(&bar_q_empty[x], (q_of[x] - 1) & 1u);
      }
      for (uint32_t u = kt < uint32_t(kStages) ? 0 : kt - kStages; u < kt; ++u) {
        const uint32_t st = u % kStages, par = (u / kStages) & 1u;
        (void)mbar_wait(&bar_k_full[st], par);
        (void)mbar_wait(&bar_v_full[st], par);
        if (ok) ok = mbar_wait(&bar_k_empty[st], par) && mbar_wait(&bar_v_empty[st], par);
      }
    } else if (warp == 17) {
      // ---------------- MMA issuer (the whole warp; see mma_ss) ----------------
      const uint32_t lead = elect_one();
      const uint32_t idesc_s = umma_idesc_f16(kBF16, 128, 128, false, false);
      const uint32_t idesc_o = umma_idesc_f16(kBF16, 128, D, false, true);
      const uint64_t dQ = umma_sdesc_sw128(smem_u32(sQ), 16, 1024), dK = umma_sdesc_sw128(smem_u32(sK), 16, 1024);
      const uint64_t dV = umma_sdesc_sw128(smem_u32(sV), kHalfBytes, 1024);
      bool ok = true;
      uint32_t kt = 0, s_of[2] = {0, 0}, q_of[2] = {0, 0}, o_of[2] = {0, 0};   // tiles; steps, Q blocks and outputs of A, B
      // S_x(t) = Q_x K_t^T into TMEM columns 128x .. 128x + 127, t of the block's `count` tiles.  A descriptor
      // advances by bytes / 16.
      auto issue_s = [&](int x, uint32_t tile, int t, int count) -> bool {
        if (t == 0 && !all(mbar_wait(&bar_q[x], q_of[x]++ & 1u))) return false;
        const uint32_t st = tile % kStages;
        if (!all(mbar_wait(&bar_k_full[st], (tile / kStages) & 1u))) return false;
        tc_fence_after();
        const uint64_t a = dQ + uint32_t(x * C::kTileBytes / 16), b = dK + uint32_t(st * C::kTileBytes / 16);
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk)
          mma_ss(lead, tmem + 128 * x, a + ((kk >> 2) * kHalfBytes + (kk & 3) * 32) / 16,
                 b + ((kk >> 2) * kHalfBytes + (kk & 3) * 32) / 16, idesc_s, kk > 0);
        commit(lead, &bar_s_full[x]);
        if (t + 1 == count) commit(lead, &bar_q_empty[x]);
        return true;
      };
      // O_x += P_x(t) V_t; P_x of each half of the keys in the first 32 columns of that half's scores.
      auto issue_pv = [&](int x, uint32_t tile, bool first) -> bool {
        const uint32_t st = tile % kStages;
        if (!all(mbar_wait(&bar_v_seen[st], (tile / kStages) & 1u))) return false;   // (long before P)
        if (first && o_of[x] > 0 && !all(mbar_wait(&bar_o_free[x], (o_of[x] - 1) & 1u))) return false;
        if (!all(mbar_wait(&bar_p_full[x], s_of[x] & 1u))) return false;
        ++s_of[x];
        tc_fence_after();
        const uint64_t b = dV + uint32_t(st * C::kTileBytes / 16);
#pragma unroll
        for (int kk = 0; kk < kTile / 16; ++kk)
          mma_ts(lead, tmem + 256 + 128 * x, tmem + 128 * x + (kk >> 2) * 64 + (kk & 3) * 8, b + kk * 2048 / 16, idesc_o,
                 !first || kk > 0);
        commit(lead, &bar_pv_done[x]);
        return true;
      };
      // One block may walk fewer tiles than the other.  A stage is released once both have read it.
      for (uint32_t i = 0; ok; ++i) {
        const Item it = take_item(i);
        if (it.na < 0) break;
        if (it.n > 0) {
          ok = (it.na == 0 || issue_s(0, kt, 0, it.na)) && (it.nb == 0 || issue_s(1, kt, 0, it.nb));
          commit(lead, &bar_k_empty[kt % kStages]);
          for (int t = 0; ok && t < it.n; ++t, ++kt) {
            if (t < it.na) ok = issue_pv(0, kt, t == 0);
            if (ok && t + 1 < it.na) ok = issue_s(0, kt + 1, t + 1, it.na);
            if (ok && t < it.nb) ok = issue_pv(1, kt, t == 0);
            commit(lead, &bar_v_empty[kt % kStages]);
            if (ok && t + 1 < it.nb) ok = issue_s(1, kt + 1, t + 1, it.nb);
            if (t + 1 < it.n) commit(lead, &bar_k_empty[(kt + 1) % kStages]);
          }
          o_of[0] += it.na > 0;
          o_of[1] += it.nb > 0;
        }
        if (kSplit) break;
        ok = ok && wait_item(i + 1);
      }
      if (!ok && lane == 0) set_error(p.err, PKV_DEVERR_TIMEOUT);
    } else if (warp >= 18) {
      // ---------------- V tiles, some of them seen in part ----------------
      bool ok = true;
      uint32_t kt = 0;
      if (first && warp == 18) {                             // the lengths, looked over once
        bool wrong = lane == 0 && (p.cu_q[0] != 0 || p.cu_k[0] != 0);
        for (int s = lane; s < p.num_seqs; s += 32) {
          const Seq q(p, s);
          wrong |= q.bad || q.Lq > p.max_q_len;
        }
        if (wrong) set_error(p.err, PKV_DEVERR_CHUNK);
      }
      for (uint32_t i = 0; ok; ++i) {
        const Item it = take_item(i);
        if (it.na < 0) break;
        for (int t = 0; ok && t < it.n; ++t, ++kt) {
          // Every tile's phase in its turn: the stage's next load waits for this tile's products, and they
          // for the arrival below.  A wait that skipped phases could take an earlier tile's for its own.
          const uint32_t st = kt % kStages;
          ok = all(mbar_wait(&bar_v_full[st], (kt / kStages) & 1u));
          if (!ok) break;
          if (it.t0 + t < it.masked) {
            if (lane == 0) mbar_arrive(&bar_v_seen[st]);
            continue;
          }
          const int kb = (it.t0 + t) * kTile;
#pragma unroll
          for (int rr = 0; rr < 2; ++rr) {
            const int r = 64 * (warp - 18) + 32 * rr + lane;
            const uint32_t vrow = smem_u32(sV + st * C::kTileBytes) + r * 128;
            if (kb + r >= it.Lk) {
#pragma unroll
              for (int c = 0; c < D / 8; ++c) sts128(vrow + c / 8 * kHalfBytes + ((c ^ r) & 7) * 16, 0u, 0u, 0u, 0u);
              continue;
            }
            uint32_t m[4] = {0, 0, 0, 0};                    // the largest magnitudes; NaN if any is
#pragma unroll
            for (int c = 0; c < D / 8; ++c) {                // (in an order without bank conflicts)
              const uint4 v = lds128(vrow + c / 8 * kHalfBytes + ((c ^ r) & 7) * 16);
              const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
              for (int u = 0; u < 4; ++u) max_magnitudes<kBF16>(m[u], w[u]);
            }
            max_magnitudes<kBF16>(m[0], m[1]);
            max_magnitudes<kBF16>(m[2], m[3]);
            max_magnitudes<kBF16>(m[0], m[2]);
            const float2 mm = unpack2<kBF16>(m[0]);
            if (fabsf(mm.x) < INFINITY && fabsf(mm.y) < INFINITY) continue;
            *static_cast<volatile int*>(&masked_item[i % (2 * kItems)]) = int(i) + 1;
            for (int c = 0; c < D / 8; ++c) {
              const uint32_t at = vrow + c / 8 * kHalfBytes + (c & 7) * 16;
              const uint4 v = lds128(at);
              uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
              for (int u = 0; u < 4; ++u) {
                const float2 f = unpack2<kBF16>(w[u]);
                if (!(fabsf(f.x) < INFINITY)) w[u] &= 0xffff0000u;
                if (!(fabsf(f.y) < INFINITY)) w[u] &= 0x0000ffffu;
              }
              sts128(at, w[0], w[1], w[2], w[3]);
            }
          }
          fence_proxy_async_smem();                            // the tile, to the tensor cores
          __syncwarp();
          if (lane == 0) mbar_arrive(&bar_v_seen[st]);
        }
        if (kSplit) break;
        ok = ok && wait_item(i + 1);
      }
      if (!ok && lane == 0) set_error(p.err, PKV_DEVERR_TIMEOUT);
    }
  }
  tc_fence_before();
  if constexpr (!kSplit) {
    __syncthreads();
  } else {
    // ---------------- combine the parts ----------------
    // Shares: `regions` rows of a block each, in the order (block 0 rows, block 1 rows).  Half a row is
    // kHalf bytes of fp32, 16-byte chunk c of row r at c ^ (r mod 8) against bank conflicts.
    const Item it = this_item();                             // (read again: uniform over the cluster)
    constexpr int kHalf = 2 * D;
    const int share = 2 * kTile / parts;                     // 128 or 64 rows
    auto rows_in = [&](int owner) -> int {                   // rows of a share that exist
      return min(share, max(0, rows_of(it, it.e0 + owner * share / kTile) - owner * share % kTile));
    };
    if (threadIdx.x == 0)
      mbar_arrive_expect_tx(&bar_recv, (parts - 1) * (rows_in(part) * 2 * kHalf + share * int(sizeof(float2))));
    __syncwarp();
    cluster_sync();                                          // every CTA's products are done: stages and Q are free
    tc_fence_after();
    if (warp < 16) {
      const int x = warp >> 3, hf = (warp >> 2) & 1, quarter = warp & 3, r = 32 * quarter + lane;
      constexpr int kODims = D / 2;                          // elements of half a row
      static_assert(2 * kTile * 2 * kHalf <= 2 * kStages * C::kTileBytes, "all rows fit in the K/V stages");
      static_assert(kTile * 2 * kHalf <= 2 * C::kTileBytes, "a share of 128 rows, or two of 64, fit in the Q area");
      const int owner = (x * kTile + 32 * quarter) / share, rr = (x * kTile + r) % share;   // rr: row of the share
      const bool any = (x == 0 ? it.na : it.nb) > 0, taken = masked_item[0] != 0;
      const int orow = query_row(it.e0 + x, r);
      const uint32_t tO = tmem + (uint32_t(32 * quarter) << 16) + 256 + 128 * x + kODims * hf;
      // Share s of this CTA's rows: [hf][row][kHalf], at 2 * share * kHalf * s in the stages.  What CTA
      // `from` sends to CTA `to` lands in its slot (from - to - 1) mod parts: slots 0 (and 1) in the Q area,
      // slot 2 in the place of its own share.
      auto slot_base = [&](int slot, int to) -> uint32_t {
        return slot < 2 ? smem_u32(sQ) + slot * 2 * share * kHalf : smem_u32(sK) + to * 2 * share * kHalf;
      };
      const uint32_t in_share = (hf * share + rr) * kHalf;   // this thread's half row in any share
      if (owner != part) {
        // ---- send: this warp's 32 half rows as soon as they are staged ----
        const bool have = any && part_ml[x][r].x != -INFINITY;   // else O holds nothing, or was never written
        const uint32_t row = smem_u32(sK) + owner * 2 * share * kHalf + in_share;
#pragma unroll
        for (int cc = 0; cc < kODims / 32; ++cc) {
          float v[32];
          if (any) {
            tmem_ld32(tO + 32 * cc, v);
            tmem_wait_ld();
          }
          if (taken) give_back(it, orow, hf, 32 * cc, v);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const uint32_t at = row + (((8 * cc + i) ^ (r & 7)) << 4);
            if (have)
              sts128(at, __float_as_uint(v[4 * i]), __float_as_uint(v[4 * i + 1]), __float_as_uint(v[4 * i + 2]),
                     __float_as_uint(v[4 * i + 3]));
            else
              sts128(at, 0u, 0u, 0u, 0u);
          }
        }
        fence_proxy_async_smem();                            // the staged rows, to the copies
        __syncwarp();
        if (lane == 0) {
          const int slot = (part - owner - 1 + parts) % parts, rr0 = rr, n32 = min(32, max(0, rows_in(owner) - rr0));
          const uint32_t bar = cluster_addr(smem_u32(&bar_recv), owner);
          if (n32 > 0)
            copy_to_cta(cluster_addr(slot_base(slot, owner) + in_share, owner), row, n32 * kHalf, bar);
          if (hf == 0)
            copy_to_cta(cluster_addr(smem_u32(&recv_ml[slot][rr0]), owner), smem_u32(&part_ml[x][32 * quarter]),
                        32 * sizeof(float2), bar);
        }
      } else {
        // ---- finish: this thread's half row from all parts ----
        const bool got = __all_sync(0xffffffffu, mbar_wait(&bar_recv, 0));
        if (!got && lane == 0) set_error(p.err, PKV_DEVERR_TIMEOUT);
        float2 ml[4];
        ml[3] = part_ml[x][r];
        float mx = ml[3].x;
#pragma unroll
        for (int s = 0; s < 3; ++s) {
          ml[s] = s + 1 < parts ? recv_ml[s][rr] : make_float2(-INFINITY, 0.f);
          mx = fmaxf(mx, ml[s].x);
        }
        float w[4], den = 0.f;
#pragma unroll
        for (int s = 0; s < 4; ++s) {
          w[s] = ml[s].x == -INFINITY ? 0.f : fast_exp2(ml[s].x - mx);
          den += w[s] * ml[s].y;
        }
        const float inv = den == 0.f ? 0.f : 1.f / den;      // (0: a row without keys; NaN stays)
        uint32_t o[kODims / 2];
#pragma unroll
        for (int cc = 0; cc < kODims / 32; ++cc) {
          float v[32];
          if (any) {
            tmem_ld32(tO + 32 * cc, v);
            tmem_wait_ld();
          }
          if (taken) give_back(it, orow, hf, 32 * cc, v);
#pragma unroll
          for (int i = 0; i < 32; ++i) v[i] = any && ml[3].x != -INFINITY ? v[i] * (w[3] * inv) : 0.f;
#pragma unroll
          for (int s = 0; s < 3; ++s) {
            if (s + 1 >= parts || !got) break;
            const uint32_t row = slot_base(s, part) + in_share;
            const float ws = w[s] * inv;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const uint4 q = lds128(row + (((8 * cc + i) ^ (r & 7)) << 4));
              v[4 * i] += ws * __uint_as_float(q.x);
              v[4 * i + 1] += ws * __uint_as_float(q.y);
              v[4 * i + 2] += ws * __uint_as_float(q.z);
              v[4 * i + 3] += ws * __uint_as_float(q.w);
            }
          }
#pragma unroll
          for (int i = 0; i < 16; ++i) o[16 * cc + i] = pack2<kBF16>(v[2 * i], v[2 * i + 1]);
        }
        if (got) write_rows(it, it.e0 + x, hf, quarter, sOut + warp * C::kOutBytes, o);
      }
    }
    __syncwarp();
    cluster_sync();                                          // every copy out of this CTA has arrived
  }
  griddep_launch_dependents();
  if (warp == 17) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

// Clusters of `parts` CTAs of the split kernel that the current device holds at once (0 on failure).
template <bool kBF16, int D, bool kPacked>
int clusters_at_once(int parts) {
  static thread_local int cached_dev = -1;
  static thread_local int cached[2];                         // parts 2 and 4
  const int dev = current_device();
  if (dev < 0) return 0;
  if (dev != cached_dev) {                                   // looked up once per device and thread
    auto kern = prompt_kernel<kBF16, D, true, kPacked>;
    for (int i = 0; i < 2; ++i) {
      cudaLaunchConfig_t cfg = {};
      cfg.gridDim = dim3(2 << i);
      cfg.blockDim = dim3(kThreads);
      cfg.dynamicSmemBytes = Cfg<D>::kSmem;
      cudaLaunchAttribute attr[1];
      attr[0].id = cudaLaunchAttributeClusterDimension;
      attr[0].val.clusterDim.x = 2 << i;
      attr[0].val.clusterDim.y = 1;
      attr[0].val.clusterDim.z = 1;
      cfg.attrs = attr;
      cfg.numAttrs = 1;
      if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg<D>::kSmem) != cudaSuccess ||
          cudaOccupancyMaxActiveClusters(&cached[i], kern, &cfg) != cudaSuccess)
        return 0;
    }
    cached_dev = dev;
  }
  return cached[parts == 2 ? 0 : 1];
}

// One item walks its keys alone unless there are so few items that clusters of 2 or 4 CTAs for each still
// run at once and every part has two key tiles or more (by the sequences' mean length).  A chunk of 512
// rows after 3584 keys (60 items of 28 heads over 4): 48.4 us alone, 33.4 us in clusters of 2; one row of 32
// heads over 8 and 4096 keys (8 items): 44.0 us alone, 17.8 us in clusters of 4.
template <bool kBF16, int D, bool kPacked>
pkv_status launch(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv, const PromptParams& prm,
                  int num_seqs, int max_q_len, cudaStream_t stream) {
  using C = Cfg<D>;
  const Blocks blocks(kPacked, prm.num_heads / prm.num_kv_heads);
  const int64_t groups = ((int64_t(max_q_len) - 1) / blocks.rows * blocks.per_tile + blocks.per_tile + 1) / 2;
  const int64_t items = groups * num_seqs * prm.num_kv_heads;
  // Items that the sequences have at most, whatever their lengths.
  const int64_t most =
      ((int64_t(prm.total_q) / blocks.rows + num_seqs + 1) * blocks.per_tile / 2 + num_seqs) * prm.num_kv_heads;
  const int64_t mean_tiles = (int64_t(prm.total_k) / num_seqs + kTile - 1) / kTile;
  int parts = 1;
  while (parts < 4 && mean_tiles >= 4 * parts && items <= clusters_at_once<kBF16, D, kPacked>(2 * parts)) parts *= 2;
  // Numbering the items level by level starts the long ones first, but has an index for every sequence
  // at every level of the longest one; past twice the items that there can be, or past what a grid
  // holds, they are numbered sequence by sequence.  One prompt of 8192 tokens among 255 of 32 (32 heads
  // over 8): 1098 us level by level, 368 us by sequence; 16 prompts of 64 to 2048 tokens (13,165 in
  // all, 28 heads over 4): 110 us and 115 us.
  const bool compact = parts == 1 && (items > 2 * most || groups > 65535);
  if (compact && most > 0x7fffffff) return PKV_ERR_UNSUPPORTED;
  PromptParams params = prm;
  params.compact = compact;
  auto kern = parts > 1 ? prompt_kernel<kBF16, D, true, kPacked> : prompt_kernel<kBF16, D, false, kPacked>;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem) != cudaSuccess)
    return PKV_ERR_CUDA;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = compact ? dim3(unsigned(most)) : dim3(unsigned(prm.num_kv_heads) * parts, num_seqs, unsigned(groups));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = C::kSmem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = unsigned(parts);
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kern, tq, tk, tv, params) == cudaSuccess ? PKV_OK : PKV_ERR_CUDA;
}

}  // namespace
}  // namespace pkv

extern "C" pkv_status pkv_prompt_attention(void* out, const void* q, const void* k, const void* v, pkv_dtype dtype,
                                           const int32_t* cu_q_lens, const int32_t* cu_k_lens, int num_seqs,
                                           int total_q, int total_k, int max_q_len, int num_heads, int num_kv_heads,
                                           int head_dim, int64_t out_stride, int64_t q_stride, int64_t k_stride,
                                           int64_t v_stride, float scale, pkv_stream_t stream) {
  using namespace pkv;
  if (num_seqs < 0 || total_q < 0 || total_k < 0 || max_q_len < 0 || num_heads <= 0 || num_kv_heads <= 0 ||
      head_dim <= 0 || num_heads % num_kv_heads)
    return PKV_ERR_INVALID_ARG;
  if (dtype != PKV_F16 && dtype != PKV_BF16) return PKV_ERR_INVALID_ARG;
  if (!(scale > 0.f)) return PKV_ERR_INVALID_ARG;            // the softmax takes max(s) * scale
  if (head_dim != 64 && head_dim != 128) return PKV_ERR_UNSUPPORTED;
  if (num_seqs > kMaxSeqs || num_heads > 65535) return PKV_ERR_UNSUPPORTED;
  // Row blocks of a sequence's kv head are numbered in 32 bits.
  if ((int64_t(max_q_len) + kTile - 1) / kTile * (num_heads / num_kv_heads) >= (int64_t(1) << 31)) return PKV_ERR_UNSUPPORTED;
  if (num_seqs == 0 || total_q == 0 || max_q_len == 0) return PKV_OK;
  if (!out || !q || !cu_q_lens || !cu_k_lens || (total_k > 0 && (!k || !v))) return PKV_ERR_INVALID_ARG;
  auto bad_rows = [&](const void* t, int64_t stride, int heads) {
    return !aligned16(t) || stride % 8 || stride < int64_t(heads) * head_dim;
  };
  if (bad_rows(out, out_stride, num_heads) || bad_rows(q, q_stride, num_heads) || bad_rows(k, k_stride, num_kv_heads) ||
      bad_rows(v, v_stride, num_kv_heads) || (reinterpret_cast<uintptr_t>(cu_q_lens) & 3u) ||
      (reinterpret_cast<uintptr_t>(cu_k_lens) & 3u))
    return PKV_ERR_INVALID_ARG;
  const int64_t kMaxStride = int64_t(1) << 38;               // a tensor map's strides end at 2^40 bytes
  if (q_stride >= kMaxStride || k_stride >= kMaxStride || v_stride >= kMaxStride) return PKV_ERR_UNSUPPORTED;
  if (!on_current_device(q) || (total_k > 0 && (!on_current_device(k) || !on_current_device(v))))
    return PKV_ERR_INVALID_ARG;
  unsigned* err = error_word_ptr();
  if (!err) return PKV_ERR_CUDA;
  // The heads of a kv head share a block unless that takes more than a sixteenth more blocks at the mean
  // length (groups that fill 128 rows badly).  Short sequences then need a fraction of the blocks, and the
  // causal border cuts off more of a block of fewer query rows.  32 sequences of 8 rows over 2048 keys, 28
  // heads over 4: 27.6 us, 99.1 with a head per block; 16 prompts of 64 to 2048 tokens: 208 us and 215; one
  // of 8192, 32 heads over 8: 322 us and 330.
  const int G = num_heads / num_kv_heads, mean = (total_q - 1) / num_seqs + 1;
  const Blocks together(true, std::min(G, kTile)), apart(false, G);
  const bool packed = G > 1 && G <= kTile &&
                      16 * int64_t((mean - 1) / together.rows + 1) <= 17 * int64_t((mean - 1) / kTile + 1) * G;
  // Rows as (dims, heads, rows): a box is 64 dims of a block's rows.
  auto encode = [&](CUtensorMap* m, const void* base, int heads, int rows, int64_t stride, const Blocks& box) {
    return encode_tmap_3d(m, CU_TENSOR_MAP_DATA_TYPE_UINT16, base, uint64_t(head_dim), uint64_t(heads), uint64_t(rows),
                          uint64_t(head_dim) * 2, uint64_t(stride) * 2, 64, box.rows == kTile ? 1 : G, box.rows,
                          CU_TENSOR_MAP_SWIZZLE_128B);
  };
  CUtensorMap tq, tk = {}, tv = {};
  if (!encode(&tq, q, num_heads, total_q, q_stride, packed ? together : apart)) return PKV_ERR_CUDA;
  if (total_k > 0 && (!encode(&tk, k, num_kv_heads, total_k, k_stride, apart) ||
                      !encode(&tv, v, num_kv_heads, total_k, v_stride, apart)))
    return PKV_ERR_CUDA;
  PromptParams prm = {.group = Divisor(G)};
  prm.out = static_cast<uint8_t*>(out);
  prm.cu_q = cu_q_lens;
  prm.cu_k = cu_k_lens;
  prm.out_stride = out_stride;
  prm.v = static_cast<const uint8_t*>(v);
  prm.v_stride = v_stride;
  prm.num_seqs = num_seqs;
  prm.compact = 0;
  prm.total_q = total_q;
  prm.total_k = total_k;
  prm.max_q_len = max_q_len;
  prm.num_heads = num_heads;
  prm.num_kv_heads = num_kv_heads;
  prm.scale_log2 = scale * 1.4426950408889634f;
  prm.err = err;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  auto run = [&](auto is_packed) -> pkv_status {
    constexpr bool kPacked = decltype(is_packed)::value;
    if (dtype == PKV_BF16)
      return head_dim == 128 ? launch<true, 128, kPacked>(tq, tk, tv, prm, num_seqs, max_q_len, s)
                             : launch<true, 64, kPacked>(tq, tk, tv, prm, num_seqs, max_q_len, s);
    return head_dim == 128 ? launch<false, 128, kPacked>(tq, tk, tv, prm, num_seqs, max_q_len, s)
                           : launch<false, 64, kPacked>(tq, tk, tv, prm, num_seqs, max_q_len, s);
  };
  return packed ? run(std::true_type{}) : run(std::false_type{});
}
