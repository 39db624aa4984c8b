// tall_kernel.cu -- attention of more than 128 query rows per KV head (prompts
// over an encoder's states, large trees of drafts), on the fifth-generation tensor
// cores.
//
// For the rows r = (t, g) of a (request, kv head), t a token and g a head of the
// group, over the keys j that rows.cuh says they see:
//     s_rj = scale q_r . k_j,   o_r = sum_j softmax(s_r)_j v_j,
// in one pass with the running maximum m and sum l: when m grows, l and o are
// scaled by 2^(m - m').  With 256 rows a key is used 256 times per read, so the
// tensor pipe bounds the kernel and not HBM, and everything else has to fit
// beside it.
//
// An item is two tiles of up to 128 rows (whole tokens: 128 / G of them each)
// over a chunk of the keys, 128 keys a step.  Per step and row tile the tensor
// core makes S = Q K^T (both from shared memory) and O += P V (P from TMEM); a
// warpgroup per row tile turns S into P.  TMEM holds S (P, in 16 bits, replaces
// its first half) and O of both tiles, all 512 columns; while one tile's S is in
// its warpgroup, the tensor core works for the other.  A tile's chain of softmax
// (about 1500 cycles), P V (514) and S (524) bounds a step at 3100 cycles, where
// the tensor core works 2080.  So: P V of the first 64 keys starts before the rest
// of P is there; the maximum is taken while the first quarter's exponentials run
// against the old one; an MMA warp elects one thread per product and folds the
// commits into it.  (64 keys a step with two buffers of S per tile, so that S is
// made ahead: slower, the smaller products cost as much as the larger.  Two
// warpgroups to a tile, half the keys each: 473 us where this took 356; the
// exponentials of a tile take about 1000 cycles of their unit whoever asks for them.)
// O is rescaled only when a row's maximum has grown by more than 2^kRaise (the
// end's division is exact about it), which is rare after the first steps.  P is
// rounded to 16 bits for the product.  Over bf16 caches O is divided by the sum of the
// weights as rounded, as in the kernels for fewer rows, so that those applied sum to
// one: the error is at most 2^-8 sum_j w_j |v_j - o|, and a row that one key dominates
// returns that key's value.  (Divided by the unrounded sum, up to 2^-8 |o| of it came
// on top.)  The second sum costs 5 to 8 % at size, with adds that take a bf16 operand;
// by unpacking P 11 %, by a warp's mma against a selection of its own lanes 40 %, and
// behind the release of P, where the warp would wait anyway, no less than before it.
// In f16 (2^-11) the unrounded sum stays; the LSE has it everywhere.
//
// The work is cut evenly, whatever the lengths: all steps of all items stand in
// one list, by pair of row tiles, request and kv head, and each CTA (one for each SM)
// takes the same share of it by measured costs (kTCostBoth).  With the pairs
// outermost, those of a (request, kv head) are worked on at about the same time and
// meet its keys in L2 (4 x 2048 tokens x 4096 keys, 32 heads with keys of their own:
// 422 us with the pairs innermost, 367 so).  At most two of a CTA's items are not
// whole; those leave fp32 partials in the CTA's two slots of the workspace, and
// tall_join_kernel merges them.  Every CTA works its share out from the lengths in
// device memory, its begin in one warp and its end in another.  (Whole items, taken
// by CTAs as they finish: 5 % faster where all lengths are equal and there are
// several items per CTA, up to twice as slow where they are not.)  Over few keys
// (a.join NULL) every cut is moved to an item's end and nothing is merged.  The copies and
// the first S of an item overlap the end of the one before.  Roles: warp 0 MMA, 1
// schedule and Q, 2-6 K and V, 8-15 softmax.  K and V go through a ring of five
// 32 KB slots (128 keys of K or of V), a warp to each; TMA boxes are of up to 128
// tokens (what divides a page).  Boxes that one warp issues are serialised (130 to
// 240 cycles), and a step of 16-token pages has 32.
// FP8 and 4-bit caches: warps 2 and 3 bring the cache's bytes to two 16 KB slots,
// warps 4-7 convert them to f16 in four operand slots (and Q's rows in place), and
// the products run in f16.  A step then takes about 3200 cycles, of which the
// converters work all: shared memory bounds it.
// Values of keys behind a sequence may be anything: they are zeroed in shared
// memory (0 x NaN is NaN).  Every wait is bounded.
//
// GB300, us in a replayed graph: 8192 tokens x 8192 keys, 32 / 8 heads: 722 to 738 as
// the clock goes (1490 to 1520 TFLOP/s, 0.79 to 0.81 of a library product's burst); 4 x
// 2048 x 4096, 32 / 8 heads: 383 to 390 (1410 to 1440); 16 requests of 4K to 16K keys,
// 256 rows per head: 137 (4.7 TB/s; a
// step is bound by HBM, 20 us are the first copies, the last output and the merge); 8
// requests of up to 448 tokens over up to 1500 FP8 states, 20 heads: 62, half of it the
// items' begins and ends (7 steps each).

#include <cfloat>
#include <mutex>
#include <type_traits>

#include "decode_attn.h"
#include "kernels.cuh"
#include "ptx.cuh"
#include "rows.cuh"
#include "tcgen05.cuh"

namespace dattn {
namespace {

constexpr float kLn2t = 0.6931471805599453f;
constexpr int kTRows = 128;                       // rows of a tile (MMA M)
constexpr int kTKeys = 128;                       // keys of a step (MMA N of S, K of P V)
constexpr int kTQHalf = kTRows * 128;             // [128 rows][64 d] bf16
constexpr int kTQTile = 2 * kTQHalf;
constexpr int kTHalf = kTKeys * 128;              // [64 tokens][64 d] bf16
constexpr int kTSlot = 2 * kTHalf;                // K or V of a step
constexpr int kTMmaWarp = 0;
constexpr int kTSchedWarp = 1;
constexpr int kTProdWarp = 2;
constexpr int kTConvWarp = 4;                     // FP8 and 4-bit caches: the second warpgroup converts
constexpr int kTConverters = 4;
constexpr int kTSoftmaxWarp = 8;                  // to 15: the last two warpgroups
constexpr int kTRawScales = 8192;                 // 4-bit caches: the block scales behind 128 keys' values
constexpr int kTThreads = 512;                    // (setmaxnreg takes whole warpgroups)
constexpr uint32_t kTTmemCols = 512;
constexpr uint32_t kTColO = 256;                  // S of tile g at 128 g, O at 256 + 128 g
// registers: 65536 / 512 threads is what the launch gives
constexpr int kTLaunchRegs = 65536 / kTThreads / 8 * 8;
constexpr int kTSoftmaxRegs = 208;
constexpr int kTOtherRegs = 48;
static_assert(256 * kTSoftmaxRegs + (kTThreads - 256) * kTOtherRegs <= kTThreads * kTLaunchRegs,
              "the register split would wait forever");

// KV: the cache's type (DA_CACHE_*).
template <int KV>
struct TCfg {
  static constexpr bool kConv = KV != DA_CACHE_BF16;       // operands are converted to f16
  static constexpr bool kFp4 = KV == DA_CACHE_FP4_E2M1;
  static constexpr int kSlots = kConv ? 4 : 5;             // operand slots: K or V of a step, 32 KB
  static constexpr int kRaw = kConv ? 2 : 0;               // slots of the cache's bytes
  static constexpr int kRawBytes = 16384;                  // 4-bit: 8 KB of values, 1 KB of scales
  // A producer warp per slot that it fills: one that filled slots in turn with
  // others could meet a slot's barrier a whole round early, where its parity says
  // "free".
  static constexpr int kProducers = kConv ? kRaw : kSlots;
  static_assert(kTProdWarp + kProducers <= (kConv ? kTConvWarp : kTSoftmaxWarp), "warps");
  static constexpr int kReaders = 8 + 1 + kProducers + (kConv ? kTConverters : 0);  // of an item's descriptor
  static constexpr int kOffRing = 2 * kTQTile;
  static constexpr int kOffRaw = kOffRing + kSlots * kTSlot;
  static constexpr int kOffBar = kOffRaw + kRaw * kRawBytes;
  static constexpr int kBars = 2 * kSlots + 2 * kRaw + 2 + 2 + 2 + 2 + 4 + 2 + 2 + 2 + 1;
  static constexpr int kOffItems = (kOffBar + kBars * 8 + 8 + 15) / 16 * 16;
  static constexpr int kOffEnd = kOffItems + 2 * 64;
  static constexpr int kOffExp = kOffEnd + 64;             // [2 items][256 rows] exponents of Q's scales
  static constexpr int kSmem = 1024 + kOffExp + (kConv ? 2 * 2 * kTRows * 2 : 0);
  static_assert(kSmem <= 227 * 1024, "shared memory");
  // P = 2^(x - m + kShift) with m the row's maximum when it was last raised; it is
  // raised when P would pass 2^(kShift + kRaise).  f16 ends at 2^16 and keeps weights
  // down to 2^-24 of 2^kShift.  bf16 holds far more, but O sums P V in fp32: with P up
  // to 2^8 (as in the kernels for fewer rows) values of up to 2^119 / keys stay finite,
  // with 2^64 those above 2^63 did not.  Raised past 8 instead of 64: no call slower
  // (GB300, 4 x 2048 tokens over 4096 keys 355 us both, 16 x 512 over 1500 107 and 109).
  static constexpr float kRaise = 8.f;                     // log2 units
  static constexpr float kShift = kConv ? 6.f : 0.f;
};

struct TallMaps {
  CUtensorMap q, k, v, ks, vs;  // (ks, vs: block scales of 4-bit caches)
};

// One piece of an item, in shared memory: written by the scheduler warp.
struct TallItem {
  int valid;             // 0: no item is left
  int b, kvh;
  int tok0;              // first token of the two row tiles
  int own, base;         // the request's own tokens, first key that goes by the mask
  int t_begin, t_end;    // keys
  int steps;
  int tiles;             // row tiles with own rows
  int slot;              // of the partials; -1: a whole item, written to out
};
static_assert(sizeof(TallItem) <= 64, "item slots");

// Costs: of a step of two row tiles (about 3000 cycles) and of one (2650: softmax,
// P V and S then follow one another), and of an item besides (Q, the first copies, the
// masked step, its output).
constexpr int kTCostBoth = kTallCostBoth, kTCostOne = 7, kTCostItem = kTallCostItem;
static_assert(kTCostOne <= kTCostBoth, "the host bounds the list's cost");
// A cut within this many steps of an item's end is moved there.
constexpr int kTSnap = 2;
// The least share: three steps.  (One whose ends are moved to the same place is empty.)
constexpr uint32_t kTCostLeast = 3 * kTCostBoth;

// The list's entries of a request.  (The host keeps the cost of the list below
// 2^32.)
struct TallRequest {
  int L, own;
  int steps;             // of an item
  int both, one;         // pairs of two row tiles with own rows, and of one (0 or 1)
  // cost of an item of pair p, and of the pairs below p, for one head
  __device__ __forceinline__ uint32_t per_step(int p) const {
    return p < both ? kTCostBoth : p == both && one != 0 ? kTCostOne : 0;
  }
  __device__ __forceinline__ uint32_t cost(int p) const {
    const uint32_t c = per_step(p);
    return steps > 0 && c > 0 ? static_cast<uint32_t>(steps) * c + kTCostItem : 0;
  }
  __device__ __forceinline__ uint32_t cost_below(int p) const {
    if (steps <= 0) return 0;
    const uint32_t n = min(p, both), n1 = p > both ? one : 0;
    return static_cast<uint32_t>(steps) * (kTCostBoth * n + kTCostOne * n1) + kTCostItem * (n + n1);
  }
  // the step of an item of pair p at cost x of it; a cut near the item's begin or end
  // (with `whole`, any) is moved there
  __device__ __forceinline__ int step_at(int p, uint32_t x, bool whole) const {
    const int s = x <= kTCostItem ? 0 : static_cast<int>((x - kTCostItem) / per_step(p));
    if (whole) return 2 * s < steps ? 0 : steps;
    return s < kTSnap ? 0 : steps - s < kTSnap ? steps : s;
  }
};

__device__ __forceinline__ TallRequest tall_request(const SplitArgs& a, int b, int tile_tokens, bool report) {
  TallRequest q;
  q.L = a.seq_lens[b];
  const int own = a.own.own_lens != nullptr ? __ldg(a.own.own_lens + b) : a.q_len;
  if (q.L < 0 || q.L > a.max_seq_len) {
    if (report && a.status != nullptr) atomicOr(a.status, static_cast<int32_t>(DA_STATUS_SEQ_LEN));
    q.L = q.L < 0 ? 0 : a.max_seq_len;
  }
  q.own = own_rows(a.own, a.q_len, b, q.L, own, report, a.status).n;
  q.steps = (q.L + kTKeys - 1) / kTKeys;
  q.both = q.own / (2 * tile_tokens);
  const int left = q.own - q.both * 2 * tile_tokens;
  q.one = left > 0 && left <= tile_tokens ? 1 : 0;
  q.both += left > tile_tokens ? 1 : 0;
  return q;
}

// The first request from b on with more than `below` rows as given (a.batch or more: there
// is none).  One thread, kTSkip loads side by side: a request at a time, a batch of 512
// (2000) of which one request has 2048 tokens and the others 1 took 1955 us (7640 us),
// now 1610 (3200); 1267 (1240) of that are the padding written as zeros.
constexpr int kTSkip = 8;
__device__ __forceinline__ int tall_skip(const SplitArgs& a, int b, int below) {
  if (a.own.own_lens == nullptr) return b;
  for (; b < a.batch; b += kTSkip) {
    uint32_t has = 0;
#pragma unroll
    for (int j = 0; j < kTSkip; ++j)
      has |= __ldg(a.own.own_lens + min(b + j, a.batch - 1)) > below ? 1u << j : 0u;
    if (has != 0) return b + __ffs(has) - 1;
  }
  return b;
}

// A place in the list: step `step` of an item (q.steps: its end).
struct TallPlace {
  int b, kvh, pair, step;
  TallRequest q;         // of request b
  uint32_t item_cost;    // cost of the list before the item
  __device__ __forceinline__ bool same_item(const TallPlace& o) const {
    return b == o.b && kvh == o.kvh && pair == o.pair;
  }
};

static_assert(sizeof(TallPlace) <= 64, "its place in shared memory");

// The cost of the list, cut into shares as even as can be: share c begins at
// begin(c).
struct TallShares {
  uint32_t total, n, each, more;  // `more` shares have one more
  __device__ __forceinline__ uint32_t begin(uint32_t c) const { return each * c + min(c, more); }
};

// The whole warp: cost of the pairs below p, for all requests.  `mine` are the
// requests of lanes 0 .. 31.
__device__ __forceinline__ uint32_t tall_cost_below(const SplitArgs& a, int tile_tokens, const TallRequest& mine, int p) {
  uint32_t sum = mine.cost_below(p);
  for (int b = 32 + (threadIdx.x & 31); b < a.batch; b += 32)
    sum += tall_request(a, b, tile_tokens, false).cost_below(p);
  return __reduce_add_sync(0xffffffffu, sum) * static_cast<uint32_t>(a.num_kv_heads);
}

// The whole warp.
__device__ __forceinline__ TallShares tall_shares(const SplitArgs& a, int tile_tokens, int pairs, bool report,
                                                  TallRequest& mine) {
  const int lane = threadIdx.x & 31;
  mine = TallRequest{};
  for (int b = lane; b < a.batch; b += 32) {
    const TallRequest q = tall_request(a, b, tile_tokens, report);
    if (b == lane) mine = q;
    else if (!report) break;  // (the others are for the status bits)
  }
  TallShares h;
  h.total = tall_cost_below(a, tile_tokens, mine, pairs);
  h.n = min(gridDim.x, max(h.total / kTCostLeast, 1u));
  h.each = h.total / h.n;
  h.more = h.total - h.each * h.n;
  return h;
}

// The whole warp: the place at cost x (below the total) of the list.
__device__ __forceinline__ TallPlace tall_place(const SplitArgs& a, int tile_tokens, int pairs, uint32_t x,
                                                const TallRequest& mine) {
  const int lane = threadIdx.x & 31;
  TallPlace p = {};
  // the last pair that begins at or before x
  uint32_t before = 0;
  int past_it = pairs;
  while (past_it - p.pair > 1) {
    const int mid = (p.pair + past_it) >> 1;
    const uint32_t c = tall_cost_below(a, tile_tokens, mine, mid);
    if (c <= x) {
      p.pair = mid;
      before = c;
    } else {
      past_it = mid;
    }
  }
  for (int b0 = 0; b0 < a.batch; b0 += 32) {
    TallRequest q = {};
    if (b0 == 0) q = mine;
    else if (b0 + lane < a.batch) q = tall_request(a, b0 + lane, tile_tokens, false);
    const uint32_t cost = q.cost(p.pair) * static_cast<uint32_t>(a.num_kv_heads);
    uint32_t upto = cost;  // inclusive scan
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t v = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += v;
    }
    const uint32_t past = __ballot_sync(0xffffffffu, before + upto > x);
    if (past != 0) {
      const int at = __ffs(past) - 1;
      p.b = b0 + at;
      p.q.L = __shfl_sync(0xffffffffu, q.L, at);
      p.q.own = __shfl_sync(0xffffffffu, q.own, at);
      p.q.steps = __shfl_sync(0xffffffffu, q.steps, at);
      p.q.both = __shfl_sync(0xffffffffu, q.both, at);
      p.q.one = __shfl_sync(0xffffffffu, q.one, at);
      before += __shfl_sync(0xffffffffu, upto - cost, at);
      break;
    }
    before += __shfl_sync(0xffffffffu, upto, 31);
  }
  const uint32_t item = p.q.cost(p.pair);
  const uint32_t kvh = (x - before) / item;
  p.kvh = static_cast<int>(kvh);
  p.item_cost = before + kvh * item;
  p.step = p.q.step_at(p.pair, x - p.item_cost, a.join == nullptr);
  return p;
}

// The rows that are in no item (of requests without keys, and of pairs of tiles that
// are all padding): a warp to a token of a request, `first` of `warps`.
__device__ __forceinline__ void zero_rows(const SplitArgs& a, int64_t first, int64_t warps) {
  const int lane = threadIdx.x & 31;
  const int tile_tokens = kTRows / a.group;
  const int64_t tokens = static_cast<int64_t>(a.batch) * a.q_len;
  for (int64_t e = first; e < tokens; e += warps) {
    const int b = static_cast<int>(e / a.q_len), t = static_cast<int>(e - static_cast<int64_t>(b) * a.q_len);
    const TallRequest q = tall_request(a, b, tile_tokens, false);
    if (q.steps > 0 && t < static_cast<int64_t>(q.both + q.one) * 2 * tile_tokens) continue;
    uint16_t* row = a.out + static_cast<int64_t>(b) * a.o_sb + static_cast<int64_t>(t) * a.o_st + lane * 4;
    for (int h = 0; h < a.num_q_heads; ++h)
      *reinterpret_cast<uint2*>(row + static_cast<int64_t>(h) * a.o_sh) = make_uint2(0u, 0u);
    for (int h = lane; h < a.num_q_heads; h += 32) a.lse[e * a.num_q_heads + h] = -INFINITY;
  }
}

// For the merge (in the workspace): the item that a CTA's share begins in the middle
// of, in n pieces, the first in share `first` (n 0: there is none).
struct TallJoin {
  int n, first, b, kvh, pair;
};
static_assert(sizeof(TallJoin) <= kTallJoinBytes, "merge records");

template <int KV>
__global__ void __launch_bounds__(kTThreads, 1)
    tall_kernel(const __grid_constant__ TallMaps maps, const SplitArgs a, const int box_tokens) {
  using C = TCfg<KV>;
  constexpr uint32_t kFull = 0xffffffffu;
  const int tid = threadIdx.x;
  const int warp = tid >> 5;
  const int lane = tid & 31;

  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint64_t* full_bar = reinterpret_cast<uint64_t*>(smem + C::kOffBar);  // [slots] operand landed (or converted)
  uint64_t* empty_bar = full_bar + C::kSlots;                         // [slots] read by the MMAs
  uint64_t* raw_full = empty_bar + C::kSlots;                         // [raw] bytes landed
  uint64_t* raw_empty = raw_full + C::kRaw;                           // [raw] converted
  uint64_t* q_full = raw_empty + C::kRaw;                             // [2] Q tile landed
  uint64_t* q_conv = q_full + 2;                                      // [2] and converted
  uint64_t* q_empty = q_conv + 2;                                     // [2] read by the item's last S
  uint64_t* s_full = q_empty + 2;                                     // [2] S in TMEM, the P V before done
  uint64_t* p_full = s_full + 2;                                      // [tile][half] 64 keys of P in TMEM
  uint64_t* o_done = p_full + 4;                                      // [2] the item's last P V
  uint64_t* item_full = o_done + 2;                                   // [2] descriptor written
  uint64_t* item_empty = item_full + 2;                               // [2] descriptor read
  uint64_t* tmem_done = item_empty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(tmem_done + 1);
  int16_t* q_exp = reinterpret_cast<int16_t*>(smem + C::kOffExp);
  auto item_slot = [&](int k) { return reinterpret_cast<TallItem*>(smem + C::kOffItems + (k & 1) * 64); };

  if (tid == 0) {
    for (int s = 0; s < C::kSlots; ++s) {
      mbar_init(&full_bar[s], C::kConv ? kTConverters : 1);
      mbar_init(&empty_bar[s], 1);
    }
    for (int s = 0; s < C::kRaw; ++s) {
      mbar_init(&raw_full[s], 1);
      mbar_init(&raw_empty[s], kTConverters);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&q_full[i], 1);
      mbar_init(&q_conv[i], kTConverters);
      mbar_init(&q_empty[i], 1);
      mbar_init(&o_done[i], 1);
      mbar_init(&s_full[i], 1);
      mbar_init(&item_full[i], 1);
      mbar_init(&item_empty[i], C::kReaders);
    }
    for (int i = 0; i < 4; ++i) mbar_init(&p_full[i], 4);
    mbar_init(tmem_done, 8);
    fence_mbar_init();
  }
  if (warp == kTMmaWarp) {
    tmem_alloc(tmem_slot, kTTmemCols);
    tmem_relinquish();
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  grid_dependency_wait();
  const uint32_t smem_base = smem_addr(smem);
  const int tile_tokens = kTRows / a.group;  // of a row tile
  auto report = [&]() {
    if (lane == 0 && a.status != nullptr) atomicOr(a.status, static_cast<int32_t>(DA_STATUS_TIMEOUT));
  };
  // Item k as every role but the scheduler gets it; false at the end, or (with
  // ok false) when the wait ran out.
  bool ok = true;
  auto next_item = [&](int k) {
    ok = __all_sync(kFull, mbar_wait(&item_full[k & 1], (k >> 1) & 1)) != 0;
    return ok && item_slot(k)->valid != 0;
  };
  auto leave_item = [&](int k) {  // its descriptor may be overwritten
    __syncwarp();
    if (lane == 0) mbar_arrive(&item_empty[k & 1]);
  };

  if (warp < kTSoftmaxWarp) {
    // The plan: the scheduler warp finds where the CTA's share begins, the MMA warp,
    // in the same code (whose instructions come once for both), where it ends.
    static_assert(kTMmaWarp < 2 && kTSchedWarp < 2, "the first two warps");
    const int cta = static_cast<int>(blockIdx.x);
    const int pairs = (a.q_len + 2 * tile_tokens - 1) / (2 * tile_tokens);
    TallShares share = {};
    TallPlace place = {};
    if (warp < 2) {
      TallRequest mine;
      share = tall_shares(a, tile_tokens, pairs, cta == 0 && warp == kTSchedWarp, mine);
      const uint32_t c = static_cast<uint32_t>(cta) + (warp == kTMmaWarp ? 1 : 0);
      if (share.total > 0 && c < share.n) place = tall_place(a, tile_tokens, pairs, share.begin(c), mine);
      if (warp == kTMmaWarp && lane == 0) *reinterpret_cast<TallPlace*>(smem + C::kOffEnd) = place;
    }
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kTOtherRegs));
    if (warp == kTSchedWarp) {
      // ===================================================== schedule, and Q
      TallPlace at = place, end = {};
      const bool some = share.total > 0 && static_cast<uint32_t>(cta) < share.n;
      const bool to_end = static_cast<uint32_t>(cta) + 1 == share.n;  // the share runs to the list's end
      asm volatile("bar.sync 1, 64;" ::: "memory");
      if (some && !to_end) end = *reinterpret_cast<const TallPlace*>(smem + C::kOffEnd);
      if (lane == 0) {
        prefetch_tensor_map(&maps.q);
        int q_use[2] = {0, 0};
        const uint32_t q_bytes = static_cast<uint32_t>(tile_tokens * a.group) * 256u;
        bool more = some;
        const TallPlace first_place = at;
        const bool begins_inside = at.step > 0 && at.step < at.q.steps;
        // the next item of the list
        auto next = [&]() {
          at.step = 0;
          if (++at.kvh < a.num_kv_heads) return;
          at.kvh = 0;
          while (true) {
            if (++at.b >= a.batch) {
              at.b = 0;
              more = ++at.pair < pairs;
            }
            if (!more) return;
            at.q = tall_request(a, at.b, tile_tokens, false);
            if (at.q.cost(at.pair) != 0) return;
            at.b = tall_skip(a, at.b + 1, at.pair * 2 * tile_tokens) - 1;
          }
        };
        if (more && at.step == at.q.steps) {
          more = to_end || !at.same_item(end);
          if (more) next();
        }
        for (int k = 0; ok; ++k) {
          TallItem it = {};
          if (more) {
            const bool last = !to_end && at.same_item(end);
            const int stop = last ? end.step : at.q.steps;
            if (stop > at.step) {
              it.valid = 1;
              it.b = at.b;
              it.kvh = at.kvh;
              it.tok0 = at.pair * 2 * tile_tokens;
              it.own = at.q.own;
              it.base = a.own.mask != nullptr ? at.q.L - at.q.own : INT_MAX;
              it.t_begin = at.step * kTKeys;
              it.t_end = min(at.q.L, stop * kTKeys);
              it.steps = stop - at.step;
              it.tiles = at.pair < at.q.both ? 2 : 1;
              it.slot = at.step > 0 ? 2 * cta : stop < at.q.steps ? 2 * cta + 1 : -1;
            }
            more = !last;
            if (more) next();
          }
          if (k > 1) ok = mbar_wait(&item_empty[k & 1], ((k >> 1) - 1) & 1);
          if (!ok) break;
          *item_slot(k) = it;
          mbar_arrive(&item_full[k & 1]);
          if (it.valid == 0) break;  // (only the last item of a share can be empty)
          if (!more) allow_dependent_launch();
#pragma unroll
          for (int g = 0; g < 2; ++g) {
            if (g >= it.tiles) break;
            if (q_use[g] > 0) ok = mbar_wait(&q_empty[g], (q_use[g] - 1) & 1);
            if (!ok) break;
            mbar_arrive_expect_tx(&q_full[g], q_bytes);
            for (int h = 0; h < 2; ++h)
              tma_load_4d_plain(smem + g * kTQTile + h * kTQHalf, &maps.q, &q_full[g], h * 64, it.kvh * a.group,
                                it.tok0 + g * tile_tokens, it.b);
            ++q_use[g];
          }
        }
        if (a.join != nullptr) {
          // the item's pieces, for the merge: its first share is the last that starts at or before its
          // first step, its last one the last that starts inside
          TallJoin join = {};
          if (some && begins_inside) {
            auto begins_at = [&](int c) {
              return first_place.q.step_at(first_place.pair, share.begin(c) - first_place.item_cost, false);
            };
            const uint32_t item_end = first_place.item_cost + first_place.q.cost(first_place.pair);
            int first = cta, past = cta + 1;
            while (first > 0 && share.begin(first) > first_place.item_cost && begins_at(first) > 0) --first;
            while (past < static_cast<int>(share.n) && share.begin(past) < item_end && begins_at(past) < first_place.q.steps)
              ++past;
            join = TallJoin{past - first, first, first_place.b, first_place.kvh, first_place.pair};
          }
          *reinterpret_cast<TallJoin*>(a.join + cta * kTallJoinBytes) = join;
        }
        if (!ok) {
          report();
#pragma unroll
          for (int g = 0; g < 2; ++g)  // no copy may still be landing when the CTA exits
            if (q_use[g] > 0) mbar_wait(&q_full[g], (q_use[g] - 1) & 1);
        }
      }
      return;
    }
    if (C::kConv && warp >= kTConvWarp) {
      // ================================================ conversion to f16
      // An E4M3 value, and a block scale times an E2M1 value, is an f16 value.  The
      // slots' layouts are those of TMA tiles in 128-byte swizzle, so that a warp's
      // loads and stores meet all banks.
      const int ct = tid - 32 * kTConvWarp;
      const int cj = ct & 7;
      int done = 0;            // units, over all items
      int q_use[2] = {0, 0};
      static_assert(!C::kConv || (C::kRaw == 2 && C::kSlots % 2 == 0), "K and V have slots of their own");
      for (int k = 0; next_item(k); ++k) {
        const int units = 2 * item_slot(k)->steps, t_begin = item_slot(k)->t_begin, t_end = item_slot(k)->t_end;
        const int tiles = item_slot(k)->tiles;
        leave_item(k);
        // a unit whose rows from `rows` on become zeros
        auto convert = [&](const uint8_t* src, uint8_t* dst, auto tail, int rows) {
          constexpr bool kTail = decltype(tail)::value;
          if constexpr (C::kFp4) {
            // 16 bytes of a row are 32 values, two whole blocks: chunks 4 (c & 1) .. + 3
            // of half c / 2
            const int c = (ct >> 3) & 3, r0 = (ct >> 5) * 8 + cj;
#pragma unroll
            for (int v = 0; v < 4; ++v) {
              const int row = r0 + 32 * v;
              const uint4 w = *reinterpret_cast<const uint4*>(src + row * 64 + ((c ^ ((cj >> 1) & 3)) << 4));
              const uint32_t s2 = e4m3x2_to_f16x2(
                  *reinterpret_cast<const uint16_t*>(src + kTRawScales + row * 8 + 2 * c));
              const uint32_t words[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                uint32_t x[4];
                e2m1x8_to_f16(words[e], x);
                const uint32_t s1 = __byte_perm(s2, 0, e < 2 ? 0x1010 : 0x3232);
#pragma unroll
                for (int q = 0; q < 4; ++q) x[q] = !kTail || row < rows ? mul_f16x2(x[q], s1) : 0u;
                *reinterpret_cast<uint4*>(dst + (c >> 1) * kTHalf + row * 128 + (((4 * (c & 1) + e) ^ cj) << 4)) =
                    make_uint4(x[0], x[1], x[2], x[3]);
              }
            }
          } else {
            // 16 bytes of a row are 16 values: chunks 2 c and 2 c + 1, of half c / 4
            const int c = (ct >> 3) & 7, r0 = (ct >> 6) * 8 + cj, c2 = (2 * c) & 7;
            const uint8_t* from = src + r0 * 128 + ((c ^ cj) << 4);
            uint8_t* to = dst + (c >> 2) * kTHalf + r0 * 128;
            const int lo_at = (c2 ^ cj) << 4, hi_at = ((c2 + 1) ^ cj) << 4;
#pragma unroll
            for (int v0 = 0; v0 < 8; v0 += 4) {
              uint4 w[4];
#pragma unroll
              for (int v = 0; v < 4; ++v) w[v] = *reinterpret_cast<const uint4*>(from + (v0 + v) * 2048);
#pragma unroll
              for (int v = 0; v < 4; ++v) {
                uint4 lo, hi;
                e4m3x4_to_f16x4(w[v].x, lo.x, lo.y);
                e4m3x4_to_f16x4(w[v].y, lo.z, lo.w);
                e4m3x4_to_f16x4(w[v].z, hi.x, hi.y);
                e4m3x4_to_f16x4(w[v].w, hi.z, hi.w);
                if (kTail && r0 + 16 * (v0 + v) >= rows) lo = hi = make_uint4(0u, 0u, 0u, 0u);
                *reinterpret_cast<uint4*>(to + (v0 + v) * 2048 + lo_at) = lo;
                *reinterpret_cast<uint4*>(to + (v0 + v) * 2048 + hi_at) = hi;
              }
            }
          }
        };
        // Q, whose tiles land before the first K; those of a later item only after
        // the last S of the one before, when its first K and V have long landed
        const int q_at = k == 0 ? 0 : 2;
        for (int e = 0; ok && e <= units; ++e) {
          if (e == q_at) {
            // Rows of Q become f16, each brought to [2^14, 2^15) by a power of two
            // (at most 2^127), which the scores are scaled back by.
#pragma unroll 1
            for (int g = 0; ok && g < tiles; ++g) {
              ok = __all_sync(kFull, mbar_wait_lazy(&q_full[g], q_use[g] & 1)) != 0;
              if (!ok) break;
              ++q_use[g];
              uint8_t* const row = smem + g * kTQTile + ct * 128;
              auto chunk = [&](int c) {
                return reinterpret_cast<uint4*>(row + (c >> 3) * kTQHalf + (((c & 7) ^ cj) << 4));
              };
              uint32_t top = 0;  // the largest magnitudes' bits (bf16 orders like integers)
#pragma unroll 4
              for (int c = 0; c < 16; ++c) {
                const uint4 v = *chunk(c);
                top = __vmaxu2(__vmaxu2(top, v.x & 0x7fff7fffu), __vmaxu2(v.y & 0x7fff7fffu, v.z & 0x7fff7fffu));
                top = __vmaxu2(top, v.w & 0x7fff7fffu);
              }
              top = max(top & 0xffffu, top >> 16);
              // (rows of zeros, or with infinities or NaN, as they are)
              const int e2 = top > 0 && top < 0x7f80u ? max(static_cast<int>(top >> 7) - 127 - 14, -127) : 0;
              const uint32_t f = static_cast<uint32_t>(127 - e2) << 7;  // 2^-e2 in bf16
              auto f16 = [&](uint32_t x) {
                const uint32_t y = mul_bf16x2(x, f | f << 16);
                return pack_f16x2(__uint_as_float(y << 16), __uint_as_float(y & 0xffff0000u));
              };
#pragma unroll 4
              for (int c = 0; c < 16; ++c) {
                uint4* const at = chunk(c);
                const uint4 v = *at;
                *at = make_uint4(f16(v.x), f16(v.y), f16(v.z), f16(v.w));
              }
              q_exp[(k & 1) * 2 * kTRows + g * kTRows + ct] = static_cast<int16_t>(e2);
              fence_proxy_async_smem();
              __syncwarp();
              if (lane == 0) mbar_arrive(&q_conv[g]);
            }
            continue;
          }
          const int u = e - (e > q_at ? 1 : 0), v = u & 1;  // K, then V
          const int os = done % C::kSlots;
          // (the phase before a slot's first use counts as complete)
          ok = mbar_wait2_warp(smem_addr(&raw_full[v]), (done >> 1) & 1, smem_addr(&empty_bar[os]),
                               (done / C::kSlots + 1) & 1);
          if (!ok) break;
          const uint8_t* src = smem + C::kOffRaw + v * C::kRawBytes;
          uint8_t* dst = smem + C::kOffRing + os * kTSlot;
          // values of keys behind the chunk's end may be anything
          const int rows = t_end - (t_begin + (u >> 1) * kTKeys);
          if (v == 1 && rows < kTKeys) convert(src, dst, std::true_type{}, rows);
          else convert(src, dst, std::false_type{}, 0);
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(&full_bar[os]);
            mbar_arrive(&raw_empty[v]);
          }
          ++done;
        }
        if (!ok) break;
      }
      if (!ok) report();
      return;
    }
    if (warp >= kTProdWarp) {
      // ====================================================== K and V copies
      // unit u (over all items): K (even) or V (odd) of a step, in the slot that this
      // warp fills.  A lane issues one box: bf16, half the d of box_tokens tokens;
      // FP8, all of them; 4-bit, values (even lanes) or block scales.
      const int pw = warp - kTProdWarp;
      if (pw >= C::kProducers) return;
      if (lane == 0 && pw == 0 && a.max_seq_len > 0) {
        prefetch_tensor_map(&maps.k);
        prefetch_tensor_map(&maps.v);
        if constexpr (C::kFp4) {
          prefetch_tensor_map(&maps.ks);
          prefetch_tensor_map(&maps.vs);
        }
      }
      uint64_t* const full = C::kConv ? raw_full : full_bar;
      uint64_t* const empty = C::kConv ? raw_empty : empty_bar;
      constexpr int kPer = KV == DA_CACHE_FP8_E4M3 ? 1 : 2;  // boxes of the same tokens
      const int boxes = kTKeys / box_tokens;
      const int half = lane & (kPer - 1);
      const int box_tok = lane / kPer * box_tokens;  // of the lane's box in the step
      // bytes of box_tokens tokens
      const uint32_t tok_bytes = static_cast<uint32_t>(box_tokens) * (C::kFp4 ? 72u : C::kConv ? 128u : 256u);
      int ubase = 0, last = -1;
      for (int k = 0; next_item(k); ++k) {
        const TallItem it = *item_slot(k);
        leave_item(k);
        const int32_t* bt_row = a.paged ? a.block_table + static_cast<int64_t>(it.b) * a.bt_stride : nullptr;
        auto page_of = [&](int u) {
          const int tok = it.t_begin + (u >> 1) * kTKeys + box_tok;  // (max_seq_len is at most 2^30)
          return bt_row != nullptr && lane < kPer * boxes && tok < it.t_end ? __ldg(bt_row + tok / a.page_size) : 0;
        };
        const int units = 2 * it.steps;
        int u = (pw - ubase) % C::kProducers;  // the warp's first unit of the item
        if (u < 0) u += C::kProducers;
        int pg_next = page_of(u);
        for (; u < units; u += C::kProducers) {
          const int use = (ubase + u) / C::kProducers;
          int pg = pg_next;
          pg_next = page_of(u + C::kProducers);
          if (use > 0) ok = __all_sync(kFull, mbar_wait_lazy(&empty[pw], (use - 1) & 1)) != 0;
          if (!ok) break;
          const int tok0 = it.t_begin + (u >> 1) * kTKeys;
          const int live = min(boxes, (it.t_end - tok0 + box_tokens - 1) / box_tokens);
          if (lane == 0) mbar_arrive_expect_tx(&full[pw], live * tok_bytes);
          __syncwarp();
          if (lane < kPer * live) {
            if (a.paged && static_cast<unsigned>(pg) >= static_cast<unsigned>(a.num_pages)) {
              if (a.status != nullptr) atomicOr(a.status, static_cast<int32_t>(DA_STATUS_BAD_PAGE));
              pg = 0;
            }
            const int tok = tok0 + box_tok;
            const int slot = a.paged ? tok % a.page_size : tok, group = a.paged ? pg : it.b;
            // (other CTAs read the same keys: no eviction hint)
            if constexpr (C::kFp4) {
              uint8_t* dst = smem + C::kOffRaw + pw * C::kRawBytes;
              if (half == 0)
                tma_load_4d_plain(dst + box_tok * 64, (u & 1) ? &maps.v : &maps.k, &full[pw], 0, it.kvh, slot, group);
              else
                tma_load_4d_plain(dst + kTRawScales + box_tok * 8, (u & 1) ? &maps.vs : &maps.ks, &full[pw], slot,
                                  it.kvh, 0, group);
            } else if constexpr (C::kConv) {
              tma_load_4d_plain(smem + C::kOffRaw + pw * C::kRawBytes + box_tok * 128, (u & 1) ? &maps.v : &maps.k,
                                &full[pw], 0, it.kvh, slot, group);
            } else {
              tma_load_4d_plain(smem + C::kOffRing + pw * kTSlot + half * kTHalf + box_tok * 128,
                                (u & 1) ? &maps.v : &maps.k, &full[pw], half * 64, it.kvh, slot, group);
            }
          }
          __syncwarp();
          last = ubase + u;
        }
        if (!ok) break;
        ubase += units;
      }
      if (!ok) {
        report();
        // no copy of this warp may still be landing when the CTA exits (without
        // a failure every one has been waited for by its readers)
        if (lane == 0 && last >= 0) mbar_wait(&full[pw], (last / C::kProducers) & 1);
      }
      return;
    }

    // ============================================================== MMA issuer
    __syncwarp();
    asm volatile("bar.arrive 1, 64;" ::: "memory");
    const uint32_t tmem = *tmem_slot;
    constexpr uint32_t kIdescS = umma_idesc_bf16(kTRows, kTKeys, false, false, C::kConv);
    constexpr uint32_t kIdescO = umma_idesc_bf16(kTRows, kHeadDim, false, true, C::kConv);
    const uint64_t q_desc = umma_smem_desc(smem_base, 16, 1024);
    const uint64_t k_desc = umma_smem_desc(smem_base + C::kOffRing, 16, 1024);
    // V [64 keys][2 x 64 d], MN-major: d halves kTHalf apart, 8-key groups 1 KB
    const uint64_t v_desc = umma_smem_desc(smem_base + C::kOffRing, kTHalf, 1024);
    // the slot and the phase parity of the next K and of the next V (units 2 i and
    // 2 i + 1 of all steps, in slots in turn)
    int k_slot = 0, v_slot = 1;
    uint32_t k_par = 0, v_par = 0;
    auto advance = [](int& slot, uint32_t& par) {
      slot += 2;
      if (slot >= C::kSlots) {
        slot -= C::kSlots;
        par ^= 1u;
      }
    };
    uint32_t par[2] = {0, 0};              // of the next step of each tile
    uint32_t q_par[2] = {0, 0};
    const uint32_t full0 = smem_addr(full_bar), empty0 = smem_addr(empty_bar), o_done0 = smem_addr(o_done), s_full0 = smem_addr(s_full), p_full0 = smem_addr(p_full);
    for (int k = 0; next_item(k); ++k) {
      const int n = item_slot(k)->steps, tiles = item_slot(k)->tiles;
      leave_item(k);
      // S of the next K for tile g; behind the last tile the slot is free, behind
      // an item's last step Q is
      auto issue_s = [&](int g, bool last_step) {
        const bool last_tile = g == tiles - 1;
        umma_bf16_ss_k128_warp<kTQHalf, kTHalf>(tmem + g * kTKeys, q_desc + static_cast<uint64_t>(g * (kTQTile >> 4)),
                                                k_desc + static_cast<uint64_t>(k_slot * (kTSlot >> 4)), kIdescS,
                                                s_full0 + 8 * g, last_tile ? empty0 + 8 * k_slot : 0u);
        if (last_step) umma_commit_warp(&q_empty[g]);
        if (last_tile) advance(k_slot, k_par);
      };
      ok = mbar_wait_warp(full0 + 8 * k_slot, k_par);
#pragma unroll
      for (int g = 0; g < 2; ++g) {
        if (!ok || g >= tiles) break;
        ok = mbar_wait_warp(smem_addr(C::kConv ? &q_conv[g] : &q_full[g]), q_par[g]);
        if (!ok) break;
        q_par[g] ^= 1u;
        tc_fence_after_sync();
        issue_s(g, n == 1);
      }
      for (int i = 0; ok && i < n; ++i) {
        const bool more = i + 1 < n;
        const uint64_t vd = v_desc + static_cast<uint64_t>(v_slot * (kTSlot >> 4));
#pragma unroll
        for (int g = 0; g < 2; ++g) {
          if (!ok || g >= tiles) break;
          const bool last_tile = g == tiles - 1;
#pragma unroll
          for (int h = 0; h < 2; ++h) {  // 64 keys of P at a time
            const uint32_t p_bar = p_full0 + 8 * (2 * g + h);
            // (a step's V and the next one's K have long landed when its first P comes)
            if (g == 0 && h == 0)
              ok = mbar_wait3_warp(full0 + 8 * v_slot, v_par, more ? full0 + 8 * k_slot : full0 + 8 * v_slot,
                                   more ? k_par : v_par, p_bar, par[g]);
            else if (ok)
              ok = mbar_wait_warp(p_bar, par[g]);
            if (!ok) break;
            tc_fence_after_sync();
            umma_bf16_ts_k64_warp<2048>(tmem + kTColO + g * kHeadDim, tmem + g * kTKeys + h * 32,
                                        vd + h * (4 * 2048 >> 4), kIdescO, i > 0 || h > 0 ? 1u : 0u,
                                        h == 0 ? 0u : last_tile ? empty0 + 8 * v_slot : more ? 0u : o_done0 + 8 * g);
          }
          if (!ok) break;
          par[g] ^= 1u;
          if (more) issue_s(g, i + 2 == n);
          else if (last_tile) umma_commit_warp(&o_done[g]);
          if (last_tile) advance(v_slot, v_par);
        }
      }
      if (!ok) break;
    }
    // TMEM is released once the softmax warps are done with it: after a failure
    // each passes at most a few waits that run out, and past ten limits it is
    // released anyway.
    const bool done = __all_sync(kFull, mbar_wait_for(tmem_done, 0, 10 * kWaitLimitNs)) != 0;
    if (!ok || !done) report();
    tc_fence_after_sync();
    tmem_dealloc(tmem, kTTmemCols);
    return;
  }

  // =================================================== softmax warpgroups
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kTSoftmaxRegs));
  const int g = (warp - kTSoftmaxWarp) >> 2;  // row tile
  const int r = tid & 127;         // its row, and the lane of TMEM
  const int rt = r / a.group;      // its token in the tile
  const bool in_tile = rt < tile_tokens;
  const uint32_t lane_base = *tmem_slot + (static_cast<uint32_t>((warp & 3) * 32) << 16);
  const uint32_t s_col = lane_base + g * kTKeys;
  const uint32_t o_col = lane_base + kTColO + g * kHeadDim;
  const bool raw = a.scale_log2 > 0.f;  // (the scores stay unscaled; the exponent's multiply-add scales)
  // Code that not every step meets is rolled up: its instructions come from L2 at
  // about a byte a cycle when they are first met.
  int ubase = 0, seq = 0, o_use = 0;
  for (int k = 0; next_item(k); ++k) {
    const TallItem& it = *item_slot(k);  // (stays in shared memory)
    const int n = it.steps;
    const int t = it.tok0 + g * tile_tokens + rt;
    const bool mine = in_tile && t < it.own;
    float m_used = -INFINITY;  // reference maximum of P (log2 domain), raised seldom
    float l = 0.f;             // sum of the weights
    float lq = 0.f;            // and of the weights as rounded into P (bf16 caches: divides O)
    const bool active = g < it.tiles;
    float sc = a.scale_log2, s_fma = raw ? sc : 1.f;
    if (active) {
      // keys below are all seen (what padding rows see does not matter: the same
      // limit for the whole CTA)
      const int t_begin = it.t_begin, t_end = it.t_end;
      const int lim = min(t_end, it.base);
      for (int i = 0; ok && i < n; ++i) {
        ok = __all_sync(kFull, mbar_wait_lazy(&s_full[g], (seq + i) & 1)) != 0;
        if (!ok) break;
        tc_fence_after_sync();
        if (C::kConv && i == 0) {  // (a row of Q is held at 2^-e of itself)
          sc = ldexpf(a.scale_log2, q_exp[(k & 1) * 2 * kTRows + g * kTRows + r]);
          if (raw) s_fma = sc = fminf(fmaxf(sc, FLT_MIN), FLT_MAX);  // (0 x -inf would be NaN)
        }
        const int tok0 = t_begin + i * kTKeys;
        const bool edge = tok0 + kTKeys > lim;
        if (edge) {
          // some key is hidden from a row, behind the chunk's end or by the mask: its
          // S becomes -inf
#pragma unroll 1
          for (int c = 0; c < kTKeys / 32; ++c) {
            float y[32];
            tmem_ld32(s_col + 32 * c, y);
            const int at = tok0 + 32 * c, left = t_end - at;
            uint32_t seen = left >= 32 ? 0xffffffffu : left > 0 ? (1u << left) - 1u : 0u;
            if (mine && seen != 0 && at + 32 > it.base) {
              const OwnRows own{it.own, it.base, a.own.mask + it.b * a.own.mask_sb, a.own.words};
              seen &= own.bits(t, at);
            }
            const float f = raw ? 1.f : sc;
            tmem_wait_ld();
#pragma unroll
            for (int w = 0; w < 2; ++w) {
              uint32_t z[16];
#pragma unroll
              for (int e = 0; e < 16; ++e)
                z[e] = __float_as_uint((seen >> (16 * w + e)) & 1u ? y[16 * w + e] * f : -INFINITY);
              tmem_st16(s_col + 32 * c + 16 * w, z);
            }
          }
          tmem_wait_st();
        }
        // P of the first quarter as if no maximum grew, while the others' S comes and
        // their maximum is taken
        const float2 s2 = make_float2(s_fma, s_fma);
        float2 ps, qs;
        uint32_t w0[16];
        auto quarter = [&](const float* x, uint32_t* w, float2 nm2) {
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const float2 y = __ffma2_rn(make_float2(x[2 * e], x[2 * e + 1]), s2, nm2);
            const float p0 = ex2(y.x);
            const float p1 = ex2(y.y);
            ps = __fadd2_rn(ps, make_float2(p0, p1));
            w[e] = C::kConv ? pack_f16x2(p0, p1) : pack_bf16x2(p0, p1);
            if constexpr (!C::kConv) add_bf16x2(qs, w[e]);
          }
        };
        auto shift = [&]() {
          const float mref = m_used == -INFINITY ? 0.f : m_used;  // (nothing seen yet: P = 0)
          return make_float2(C::kShift - mref, C::kShift - mref);
        };
        float x[kTKeys];
        {
          float y[4][32];
#pragma unroll
          for (int c = 0; c < 4; ++c) tmem_ld32(s_col + 32 * c, y[c]);
          tmem_wait_ld();
#pragma unroll
          for (int e = 0; e < 32; ++e) x[e] = !raw && !edge ? y[0][e] * sc : y[0][e];
          ps = qs = make_float2(0.f, 0.f);
          quarter(x, w0, shift());
#pragma unroll
          for (int e = 32; e < kTKeys; ++e) x[e] = y[e / 32][e % 32];
        }
        if (!raw && !edge) {
#pragma unroll
          for (int e = 32; e < kTKeys; ++e) x[e] *= sc;
        }
        float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int e = 0; e < kTKeys; e += 8)
#pragma unroll
          for (int c = 0; c < 4; ++c) mx[c] = fmax3(mx[c], x[e + 2 * c], x[e + 2 * c + 1]);
        const float mt = fmax3(fmaxf(mx[0], mx[1]), mx[2], mx[3]) * s_fma;
        const bool raise = mt > m_used + C::kRaise;  // (from -inf by anything that is seen)
        if (__any_sync(kFull, raise)) {
          const float alpha = raise ? ex2(m_used - mt) : 1.f;
          if (raise) m_used = mt;
          l *= alpha;
          lq *= alpha;
          if (i > 0) {  // (S of this step is complete, so is the P V issued before it)
#pragma unroll 1
            for (int c = 0; c < kHeadDim / 16; ++c) {
              float o[16];
              tmem_ld16(o_col + c * 16, o);
              tmem_wait_ld();
              uint32_t w[16];
#pragma unroll
              for (int e = 0; e < 16; ++e) w[e] = __float_as_uint(o[e] * alpha);
              tmem_st16(o_col + c * 16, w);
            }
          }
          ps = qs = make_float2(0.f, 0.f);
          quarter(x, w0, shift());
        }
        const float2 nm2 = shift();
        const int n_valid = t_end - tok0;
        auto p_ready = [&](int h) {
          tmem_wait_st();
          tc_fence_before_sync();
          __syncwarp();
          if (lane == 0) mbar_arrive(&p_full[2 * g + h]);
        };
        // values of keys behind the chunk's end are zeroed before the first P V
        // (that of tile 0) may read them
        if (!C::kConv && g == 0 && n_valid < kTKeys) {
          const int u = ubase + 2 * i + 1;
          ok = __all_sync(kFull, mbar_wait_lazy(&full_bar[u % C::kSlots], (u / C::kSlots) & 1)) != 0;
          if (!ok) break;
          uint8_t* vs = smem + C::kOffRing + (u % C::kSlots) * kTSlot;
          for (int z = r; z < (kTKeys - n_valid) * 16; z += 128)
            *reinterpret_cast<uint4*>(vs + ((z >> 3) & 1) * kTHalf + (n_valid + (z >> 4)) * 128 + (z & 7) * 16) =
                make_uint4(0u, 0u, 0u, 0u);
          fence_proxy_async_smem();
        }
        tmem_st16(s_col, w0);
#pragma unroll
        for (int c = 1; c < 4; ++c) {
          uint32_t w[16];
          quarter(x + 32 * c, w, nm2);
          if (c == 2) {
            // the first half has been stored meanwhile; the last quarter stays
            // behind its release (the compiler would take it first)
            p_ready(0);
#pragma unroll
            for (int e = 96; e < 128; e += 8)
              asm volatile("" : "+f"(x[e]), "+f"(x[e + 1]), "+f"(x[e + 2]), "+f"(x[e + 3]), "+f"(x[e + 4]), "+f"(x[e + 5]),
                           "+f"(x[e + 6]), "+f"(x[e + 7]));
          }
          tmem_st16(s_col + 16 * c, w);
        }
        p_ready(1);
        l += ps.x + ps.y;
        lq += qs.x + qs.y;
      }
      if (ok) {
        ok = __all_sync(kFull, mbar_wait_lazy(&o_done[g], o_use & 1)) != 0;
        tc_fence_after_sync();
      }
      seq += n;
      ++o_use;
    }
    ubase += 2 * n;

    // ---- the rows' outputs.  A lane holds 16 columns of its row at a time; two lanes
    // trade, so that they write 32 bytes, a sector, of one of their rows and then of
    // the other (16 bytes of each row at a time take longer, and more instructions do:
    // they are met once an item)
    const bool direct = it.slot < 0;
    const bool writes = in_tile && t < a.q_len;
    const int h = it.kvh * a.group + (r - rt * a.group);
    const int64_t prow = (static_cast<int64_t>(it.b) * a.q_len + t) * a.num_q_heads + h;
    const int64_t pidx = static_cast<int64_t>(it.slot) * (2 * kTRows) + g * kTRows + r;
    const bool have = ok && active && mine && l != 0.f;
    const float inv = have ? (1.f / (C::kConv ? l : lq)) * a.v_scale : 0.f;  // (NaN stays NaN)
    // byte offset of the row, -1 where nothing is written
    const int64_t row_at = !writes ? -1
                           : direct ? 2 * (static_cast<int64_t>(it.b) * a.o_sb + static_cast<int64_t>(t) * a.o_st +
                                           static_cast<int64_t>(h) * a.o_sh)
                                    : 4 * kHeadDim * pidx;
    if (writes) {
      const float lse = !have ? -INFINITY : (m_used == -INFINITY ? 0.f : m_used - C::kShift) * kLn2t + logf(l);
      if (direct) a.lse[prow] = lse;
      else a.part_lse[pidx] = lse;
    }
    uint8_t* const dst = direct ? reinterpret_cast<uint8_t*>(a.out) : reinterpret_cast<uint8_t*>(a.part_o);
    // (rolled up: the code is met once an item, and its first pass waits for the
    // instructions)
    const bool odd = (lane & 1) != 0;
    const int64_t pair_at = __shfl_xor_sync(kFull, row_at, 1);
    const int64_t at0 = odd ? pair_at : row_at, at1 = odd ? row_at : pair_at;  // of the even and the odd lane's row
    auto write = [&](const uint32_t (&w)[8], int offset) {
      uint32_t got[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) got[e] = __shfl_xor_sync(kFull, odd ? w[e] : w[4 + e], 1);
      uint8_t* const to = dst + offset + (odd ? 16 : 0);
      if (at0 >= 0)
        *reinterpret_cast<uint4*>(to + at0) =
            odd ? make_uint4(got[0], got[1], got[2], got[3]) : make_uint4(w[0], w[1], w[2], w[3]);
      if (at1 >= 0)
        *reinterpret_cast<uint4*>(to + at1) =
            odd ? make_uint4(w[4], w[5], w[6], w[7]) : make_uint4(got[0], got[1], got[2], got[3]);
    };
#pragma unroll 1
    for (int c = 0; c < kHeadDim / 16; ++c) {
      float o[16];
      if (active) {
        tmem_ld16(o_col + c * 16, o);
        tmem_wait_ld();
      }
      if (direct) {
        uint32_t w[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) w[e] = have ? pack_bf16x2(o[2 * e] * inv, o[2 * e + 1] * inv) : 0u;
        write(w, c * 32);
      } else {
#pragma unroll
        for (int d = 0; d < 2; ++d) {
          uint32_t w[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) w[e] = have ? __float_as_uint(o[8 * d + e] * inv) : 0u;
          write(w, c * 64 + d * 32);
        }
      }
    }
    leave_item(k);
    // O was read before this warp's next P, which the next item's P V waits for
    tc_fence_before_sync();
    if (!ok) break;
  }
  if (!ok) report();
  tc_fence_before_sync();
  __syncwarp();
  if (lane == 0) mbar_arrive(tmem_done);
  if (a.join == nullptr)  // (no merge follows)
    zero_rows(a, static_cast<int64_t>(warp - kTSoftmaxWarp) * gridDim.x + blockIdx.x, 8 * static_cast<int64_t>(gridDim.x));
}

// Merges the pieces of items: piece 0 in slot 2 j + 1 of the CTA j that began it, the
// others in slots 2 (j + 1), 2 (j + 2), ..; half a warp per row, 8 d a lane.
//     M = max_s lse_s,  w_s = exp(lse_s - M),  out = sum w_s O_s / sum w_s,
// kJoinAhead pieces at a time.  The blocks blockIdx.x of all CTAs with a later piece
// share the item's rows.  It also writes the rows that are in no item.
// What bounds it is the latency of the chain (record, pieces, output) and, with a
// warp per row, was the number of instructions.
constexpr int kJoinWarps = 8;
constexpr int kJoinBlocks = 4;                    // of a piece: all blocks are on the SMs together
constexpr int kJoinAhead = 4;

__global__ void __launch_bounds__(32 * kJoinWarps, kJoinBlocks) tall_join_kernel(const SplitArgs a) {
  constexpr float kLog2e = 1.4426950408889634f;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int tile_tokens = kTRows / a.group;
  // ---- the item's share of this block
  grid_dependency_wait();
  const TallJoin join = *reinterpret_cast<const TallJoin*>(a.join + blockIdx.x * kTallJoinBytes);
  const int n = join.n;
  const int share = (static_cast<int>(blockIdx.x) - join.first - 1) * kJoinBlocks + static_cast<int>(blockIdx.y);
  const int sub = lane & 15;
  constexpr int64_t kSlotLse = 2 * kTRows, kSlotO = kSlotLse * kHeadDim;
  for (int row = (share * kJoinWarps + warp) * 2 + (lane >> 4); n > 0 && row < 2 * kTRows;
       row += (n - 1) * kJoinBlocks * kJoinWarps * 2) {
    const int g = row / kTRows, r = row - g * kTRows, rt = r / a.group;
    const int t = join.pair * 2 * tile_tokens + g * tile_tokens + rt;
    if (rt >= tile_tokens || t >= a.q_len) continue;
    const int h = join.kvh * a.group + (r - rt * a.group);
    // piece s >= 1 is 2 s slots further than this
    const float* const lses = a.part_lse + row + 2 * join.first * kSlotLse;
    const float* const parts = a.part_o + row * kHeadDim + sub * 8 + 2 * join.first * kSlotO;
    float M = -INFINITY, W = 0.f;
    float acc[8] = {};
    for (int s0 = 0; s0 < n; s0 += kJoinAhead) {
      float l[kJoinAhead];
      float4 x[kJoinAhead][2];
#pragma unroll
      for (int e = 0; e < kJoinAhead; ++e) {
        const int at = s0 + e == 0 ? 1 : 2 * (s0 + e);
        const bool have = s0 + e < n;
        l[e] = have ? lses[at * kSlotLse] : -INFINITY;
        const float4* from = reinterpret_cast<const float4*>(parts + at * kSlotO);
        x[e][0] = have ? from[0] : make_float4(0.f, 0.f, 0.f, 0.f);
        x[e][1] = have ? from[1] : make_float4(0.f, 0.f, 0.f, 0.f);
      }
      float m = M;
#pragma unroll
      for (int e = 0; e < kJoinAhead; ++e) m = fmax_nan(m, l[e]);
      const float ref = m == -INFINITY ? 0.f : m;
      const float alpha = ex2((M - ref) * kLog2e);
      M = m;
      W *= alpha;
#pragma unroll
      for (int d = 0; d < 8; ++d) acc[d] *= alpha;
#pragma unroll
      for (int e = 0; e < kJoinAhead; ++e) {
        const float w = ex2((l[e] - ref) * kLog2e);
        const float y[8] = {x[e][0].x, x[e][0].y, x[e][0].z, x[e][0].w, x[e][1].x, x[e][1].y, x[e][1].z, x[e][1].w};
        W += w;
#pragma unroll
        for (int d = 0; d < 8; ++d) acc[d] += w * y[d];
      }
    }
    const float inv = W == 0.f ? 0.f : 1.f / W;
    *reinterpret_cast<uint4*>(a.out + static_cast<int64_t>(join.b) * a.o_sb + static_cast<int64_t>(t) * a.o_st +
                              static_cast<int64_t>(h) * a.o_sh + sub * 8) =
        make_uint4(pack_bf16x2(acc[0] * inv, acc[1] * inv), pack_bf16x2(acc[2] * inv, acc[3] * inv),
                   pack_bf16x2(acc[4] * inv, acc[5] * inv), pack_bf16x2(acc[6] * inv, acc[7] * inv));
    if (sub == 0)
      a.lse[(static_cast<int64_t>(join.b) * a.q_len + t) * a.num_q_heads + h] = W == 0.f ? -INFINITY : M + logf(W);
  }
  zero_rows(a, (static_cast<int64_t>(blockIdx.y) * gridDim.x + blockIdx.x) * kJoinWarps + warp,
            static_cast<int64_t>(gridDim.x) * gridDim.y * kJoinWarps);
}

std::mutex g_tall_mu;
bool g_tall_attr[3][64];

template <int KV>
cudaError_t launch_tall_t(const TallMaps& maps, const SplitArgs& a, int box_tokens, int ctas, cudaStream_t stream) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  {
    std::lock_guard<std::mutex> lk(g_tall_mu);
    if (!g_tall_attr[KV][dev]) {
      e = cudaFuncSetAttribute(tall_kernel<KV>, cudaFuncAttributeMaxDynamicSharedMemorySize, TCfg<KV>::kSmem);
      if (e != cudaSuccess) return e;
      g_tall_attr[KV][dev] = true;
    }
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(ctas));
  cfg.blockDim = dim3(kTThreads);
  cfg.dynamicSmemBytes = TCfg<KV>::kSmem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, tall_kernel<KV>, maps, a, box_tokens);
  if (e != cudaSuccess || a.join == nullptr) return e;
  cfg.gridDim = dim3(static_cast<unsigned>(ctas), kJoinBlocks);
  cfg.blockDim = dim3(32 * kJoinWarps);
  cfg.dynamicSmemBytes = 0;
  return cudaLaunchKernelEx(&cfg, tall_join_kernel, a);
}

}  // namespace

int tall_tile_tokens(int group) { return kTRows / group; }

cudaError_t launch_tall(int type, const CUtensorMap& q_map, const Fp4Maps& kv, const SplitArgs& a, int box_tokens,
                        int sm_count, cudaStream_t stream) {
  const int ctas = sm_count < kTallCtas ? sm_count : kTallCtas;
  const TallMaps maps{q_map, kv.k, kv.v, kv.ks, kv.vs};
  switch (type) {
    case DA_CACHE_BF16: return launch_tall_t<DA_CACHE_BF16>(maps, a, box_tokens, ctas, stream);
    case DA_CACHE_FP8_E4M3: return launch_tall_t<DA_CACHE_FP8_E4M3>(maps, a, box_tokens, ctas, stream);
    default: return launch_tall_t<DA_CACHE_FP4_E2M1>(maps, a, box_tokens, ctas, stream);
  }
}

}  // namespace dattn
