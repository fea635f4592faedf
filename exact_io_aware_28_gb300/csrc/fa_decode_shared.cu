// Decode attention over a paged cache for groups of sequences that share a prefix: one new query
// token per sequence, the keys and values of a group's shared tokens read once for all of it.
//
// Mathematics.  A sequence's keys are its group's shared ones, j < S, and its own, S <= j < L:
//   o = (sum over the parts i of 2^(m_i - M) o_i) / (sum of 2^(m_i - M) l_i),
// with each part's maximum m_i, sum l_i and unnormalised o_i in fp32 (log2 domain, c = scale
// log2 e).  Over the shared keys the group's queries of one key/value head are the rows of one
// matrix product, as in a prompt, up to 256 rows a CTA; over its own keys a sequence is what it is
// in fa_decode_paged.cu.  P is rounded once to bf16 as an operand of P V in both.
//
// What bounds it: the bytes of the prefixes, once, and of the continuations; with many sequences a
// group also the products over the prefix, 4 S d operations a row, on the tensor cores.  (A group of
// more than 256 rows a head reads its prefix from DRAM more often where the cut sets the pieces apart
// in time: 256 sequences behind 16384 tokens with 128 of their own 350 MB for 201; set side by side by
// other costs of the tiles they read 218, and the call took 94 us for 91.)  Measured
// (32 / 8 heads, d = 128): 64 sequences, 8192 shared tokens and 512 of their own, pages of 64, 43 us
// for 25 us of bytes (fa_decode_paged, with the prefix from L2 for all but the first, 173); 256
// sequences, 32768 shared, pages of 128, 118 us for 72 us of operations.  A prefix tile with all 256
// rows is a chain of 1.8 to 2 us, as in the forward kernel, 1.0 to 1.2 us with rows for one tile at
// d = 64; 10 us do not grow with the lengths: lengths, tables and the first tiles 5, the join 5.
//
// Work.  The tiles of 128 keys of all prefixes lie on one line (group by group, head by head, 256
// rows by 256 rows), those of the continuations on another (sequence by sequence, head by head).
// The CTAs, one an SM, are shared out between the two by what the tiles cost, and worker w of a
// line's W takes its tiles [total w / W, total (w + 1) / W): both kinds run side by side, products of
// the one beside loads of the other, and end at about the same time.  Every segment of a pair in a
// worker's range leaves a partial result in a place of its own: (pair) + (worker) grows along the
// line, so no two meet.  A combine kernel joins them.  The cut depends on lengths, groups and the
// number of SMs alone: the same call gives the same bits.  Which kernels run depends on the width of
// the table too (decode_apart): another width may give the same batch other bits.
//
// A prefix segment (one CTA, two tiles of up to 128 query rows; a tile holds 128 / G sequences of
// G heads, in whole sequences):
//   warps 0, 2 producers of keys and values (a lane per page); warps 1, 3 MMA issuers, one a tile;
//   warps 4-11 softmax, all of them on each tile in turn: S = Q K^T in tensor memory, P over it as
//   bf16, O += P V.  A group with rows for one tile only has its queries in both, and the two take
//   the key tiles in turn.
// A sequence shorter than its group's shared tokens takes no part in them: it reads its own keys
// from the first on, and the products it is in are never joined.  Pages outside the pool are holes,
// as in fa_decode_paged.cu: not loaded, their scores replaced, their V rows zeroed.
// With few tiles for each SM the sequences are decoded apart, by fa_decode_paged.cu (decode_apart).
// Every wait is bounded; on expiry the CTA records FA_ERR_TIMEOUT and leaves.
#include <atomic>

#include <cuda.h>
#include <cudaTypedefs.h>
#include <math.h>

#include "fa_decode_units.cuh"
#include "fa_internal.cuh"
#include "fa_paged_sched.cuh"
#include "sm103_ptx.cuh"

namespace fa {
namespace {

using namespace decode;

constexpr int kRows = 128;                       // query rows of a tile

template <int D>
struct PC {
  static constexpr int NSUB = D / 64;
  static constexpr int TILE = NSUB * kSub;
  // Stages of keys and of values (three and two of them at d = 128, with the barriers moved out of
  // the tiles' way: 121 against 122 us for 256 sequences behind 32768 tokens, and 39 against 35 for
  // continuations alone).
  static constexpr int NK = D == 128 ? 2 : 4, NV = NK;
  static constexpr int TILES = (2 + NK + NV) * TILE;
  // A CTA has the memory that one on continuations has.
  static_assert(TILES <= TC<D>::STAGES * TC<D>::STAGE, "the continuations' barriers lie behind");
};
constexpr int kSeen = 8;                         // row masks of the last key tiles

struct PBars {
  uint64_t q_full, q_empty;
  uint64_t k_full[4], k_empty[4], v_full[4], v_empty[4];
  uint64_t s_full[2], p_full[2], o_done[2], o_empty[2];
  uint64_t drain;
  uint32_t seen[kSeen];
  uint32_t tmem_base;
  int abort;
  int never;
};

struct SharedArgs {
  PagedArgs a;                 // of the continuations; a.part their partial results
  const int32_t* start;        // [groups + 1]
  const int32_t* len;          // [groups]
  int groups;
  int seqs;                    // sequences of a tile: 128 / G
  // Of the prefixes: unnormalised o [entries][D], maximum and sum [entries].  Rows of whole sectors:
  // the stores of a piece's 256 rows stall on any other.
  float* part;
  float2* stats;
  int entries;
  struct Row* rows;            // [B], for the combine kernel
  struct Line* line;
  int* tiles_g;                // [groups], tiles before each group
};

// What the combine kernel needs to know of a sequence: where on the line its own tiles and its
// piece's begin (head 0), and the places of its partial results.
struct Row {
  int own, pre;
  int pre_head;                // from a head's tiles of the piece to the next head's
  int entry;                   // place of the row of head 0 in the prefixes' results
  int n;                       // own tiles of a head
  int span;                    // from the piece's first tile to its last; -1: nothing shared
  int entry_head;              // from one head's places to the next one's
  int pad;
};
struct Line {
  int total[2];                // tiles of the prefixes, of the continuations
  int workers[2];              // that have a range
};

__device__ __forceinline__ int cap_of(const PagedArgs& a) { return a.max_pages << a.page_shift; }

// The arguments with the lists of lengths and groups: copies in shared memory where they fit (what
// the tiles leave of it).
constexpr int kListed = 150;
struct Lists {
  int32_t cache_len[kListed], len[kListed], start[kListed + 1];
};
struct Plan {
  const SharedArgs& s;
  const PagedArgs& a;
  const int32_t *cache_len, *len, *start;
  int groups, seqs;
  // By all threads; before the block's barrier.
  __device__ __forceinline__ Plan(const SharedArgs& g, Lists* lists)
      : s(g), a(g.a), cache_len(g.a.cache_len), len(g.len), start(g.start), groups(g.groups),
        seqs(g.seqs) {
    if (a.B > kListed) return;                   // groups <= B
    const int i = threadIdx.x;
    if (i < a.B) lists->cache_len[i] = cache_len[i];
    if (i < groups) lists->len[i] = len[i], lists->start[i] = start[i];
    if (i == 0) lists->start[groups] = start[groups];
    cache_len = lists->cache_len;
    len = lists->len;
    start = lists->start;
  }
};

// floor(total w / workers) and the worker whose range holds x, in 32 bits: with total = q workers + r
// the first is q w + floor(r w / workers), workers being SMs (r w fits); the second is a quotient in
// fp32, off by one at most.
__device__ __forceinline__ int range_start(int total, int w, int workers) {
  const int q = total / workers;
  return q * w + (total - q * workers) * w / workers;
}
__device__ __forceinline__ int owner(int x, int total, int workers) {
  int w = static_cast<int>(static_cast<float>(x) * static_cast<float>(workers) /
                           static_cast<float>(total));
  w = min(w, workers - 1);
  if (range_start(total, w, workers) > x) --w;
  else if (w + 1 < workers && range_start(total, w + 1, workers) <= x) ++w;
  return w;
}

// What a tile costs, in some 0.3 us: a prefix's with rows for both row tiles, for one; a
// continuation's; what a pair adds to its tiles (queries, results): a prefix's, a continuation's; and
// what a prefix's CTA takes more than another, however few its tiles are.  (Mean over 28 shapes drawn
// from 16 to 256 sequences in groups of 4 to 256, prefixes of 1024 to 32768 and up to 1024 own tokens:
// 39.05 us; with 6 and 24 for the first and the last 39.23, 6 and 28 39.98, 7 and 28 40.3, 7 and 32
// 40.4, a continuation's pair at 4 39.6, at 2 40.1.)
constexpr int kCostBoth = 7, kCostOne = 4, kCostOwn = 4, kCostPrefixPair = 4, kCostOwnPair = 3;
constexpr int kCostPrefixMore = 20;
// What the prefixes cost with ascending starts, whose tiles are fewer than 2^29 (and pairs no more than
// tiles), with room for the rounding of the sum; below it the tiles of any starts fit in 32 bits.
constexpr float kMostCost = 1.1f * (kCostBoth + kCostPrefixPair) * 0x1p29f;
static_assert(kCostOne <= kCostBoth && kMostCost < kCostOne * 0x1p31f, "tiles in 32 bits");

struct Group {
  int s0, s1;                  // its sequences
  int len;                     // shared tokens; shorter sequences take no part
  int keys;                    // of them, those read once: whole boxes
  int supers;                  // pieces of up to 2 x seqs sequences
  int tiles;
  int cost;                    // of a tile
  __device__ __forceinline__ Group(const Plan& g, int p) {
    s0 = min(max(g.start[p], 0), g.a.B);
    s1 = max(s0, min(max(g.start[p + 1], 0), g.a.B));
    const int box = min(kBox, 1 << g.a.page_shift);
    // one sequence alone shares with nobody
    len = s1 - s0 > 1 ? sched::clamp_len(g.len, p, cap_of(g.a)) : 0;
    keys = len & ~(box - 1);
    supers = (s1 - s0 + 2 * g.seqs - 1) / (2 * g.seqs);
    tiles = sched::granules<kKeys>(keys);
    cost = s1 - s0 > g.seqs ? kCostBoth : kCostOne;
  }
  // Its tiles of all heads and pieces.
  __device__ __forceinline__ int all(const Plan& g) const {
    return tiles * g.a.Hkv * supers;
  }
};

// The group of sequence b: the last whose first sequence is not behind it.
__device__ __forceinline__ int group_at(const Plan& g, int b) {
  int lo = 0, hi = g.groups;
#pragma unroll 1
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (g.start[mid] <= b) lo = mid; else hi = mid;
  }
  return lo;
}

// Tokens of sequence b (length L) that it takes from its group.
__device__ __forceinline__ int shared_of(const Plan& g, const Group& p, int b, int L) {
  return b >= p.s0 && b < p.s1 && L >= p.len ? p.keys : 0;
}

struct SharedStart {
  int mine;                    // 0: the CTA works on prefixes, 1: on continuations
  int w;                       // which of their workers it is
  int first, last;             // its range of their tiles
  int p, b, pb;                // group of the first tile; sequence of the first tile, and its group
  int before;                  // tiles before that group or sequence
};

// How many of W workers go to the prefixes: so many, n, that both kinds end at the same time,
//   cost_g / n + D = cost_b / (W - n),   D = kCostPrefixMore,
// and none that one kind has no tile for while the other has.  The two SMs of a pair (the CTAs 2 i and
// 2 i + 1) do the same: with one on a prefix and one on continuations both take up to twice as long
// (16 groups of 4 sequences, 2048 + 128 tokens, so mixed throughout: 81 us against 47; the cause is
// not known).
__device__ __forceinline__ int prefix_workers(int W, int tiles_g, int tiles_b, float cost_g,
                                              float cost_b) {
  if (tiles_g == 0 || tiles_b == 0) return tiles_g == 0 ? 0 : W;
  if (tiles_g + tiles_b <= W) return static_cast<int>(tiles_g);
  const float D = kCostPrefixMore, p = D * W - cost_g - cost_b;
  int n = static_cast<int>((p + sqrtf(p * p + 4.f * D * cost_g * W)) / (2.f * D) + 0.5f);
  n += 2 * n <= W ? n & 1 : -(n & 1);
  n = max(min(n, tiles_g), W - tiles_b);
  return max(1, min(W - 1, n));
}

struct Sums {
  int tiles[2];
  float cost[2];
};

// The CTA's part of the work, as sched::find_start; block 0 writes what the combine kernel reads.
__device__ __forceinline__ void find_start(SharedStart* out, Sums* scratch,
                                           const Plan& g) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, B = g.a.B, cap = cap_of(g.a);
  const int per_p = (g.groups + kThreads - 1) / kThreads, per_b = (B + kThreads - 1) / kThreads;
  const int p0 = min(tid * per_p, g.groups), p1 = min(p0 + per_p, g.groups);
  const int b0 = min(tid * per_b, B), b1 = min(b0 + per_b, B);
  const int at0 = b0 < b1 ? group_at(g, b0) : 0;
  auto own_tiles = [&](int b, int* p) {        // of a head
#pragma unroll 1
    while (*p + 1 < g.groups && g.start[*p + 1] <= b) ++*p;
    const int L = sched::clamp_len(g.cache_len, b, cap);
    const Group gr(g, *p);
    return sched::granules<kKeys>(L - shared_of(g, gr, b, L));
  };
  int sum[2] = {0, 0};
  float cost[2] = {0.f, 0.f};
#pragma unroll 1
  for (int p = p0; p < p1; ++p) {
    const Group gr(g, p);
    sum[0] += gr.all(g);
    if (gr.tiles > 0)
      cost[0] += static_cast<float>(gr.tiles * gr.cost + kCostPrefixPair) *
                 static_cast<float>(g.a.Hkv * gr.supers);
  }
  {
    int p = at0;
#pragma unroll 1
    for (int b = b0; b < b1; ++b) {
      const int n = own_tiles(b, &p);
      sum[1] += n * g.a.Hkv;
      if (n > 0) cost[1] += static_cast<float>(n * kCostOwn + kCostOwnPair) * g.a.Hkv;
    }
  }
  int incl[2] = {sum[0], sum[1]};
#pragma unroll
  for (int off = 1; off < 32; off <<= 1)
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int up = __shfl_up_sync(0xffffffffu, incl[i], off);
      if (lane >= off) incl[i] += up;
    }
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) {
    cost[0] += __shfl_xor_sync(0xffffffffu, cost[0], off);
    cost[1] += __shfl_xor_sync(0xffffffffu, cost[1], off);
  }
  if (lane == 31) scratch[warp] = Sums{{incl[0], incl[1]}, {cost[0], cost[1]}};
  __syncthreads();
  int before[2] = {incl[0] - sum[0], incl[1] - sum[1]}, total[2] = {0, 0};
  cost[0] = cost[1] = 0.f;
#pragma unroll
  for (int i = 0; i < kThreads / 32; ++i) {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int v = scratch[i].tiles[j];
      if (i < warp) before[j] += v;
      total[j] += v;
      cost[j] += scratch[i].cost[j];
    }
  }
  // Group starts that are not ascending can name more tiles than 32 bits hold: nothing is done then.
  if (cost[0] > kMostCost) total[0] = total[1] = 0;
  const int share = prefix_workers(gridDim.x, total[0], total[1], cost[0], cost[1]);
  const int W0 = sched::active(total[0], share);
  const int W1 = sched::active(total[1], static_cast<int>(gridDim.x) - share);
  const int block = blockIdx.x, mine = block < share ? 0 : 1, w = block - (mine ? share : 0);
  const int W = mine ? W1 : W0;
  const int all = mine ? total[1] : total[0];
  const bool works = w < W;
  const int first = works ? range_start(all, w, W) : 0;
  if (tid == 0) {
    out->mine = mine;
    out->w = w;
    out->first = first;
    out->last = works ? range_start(all, w + 1, W) : 0;
  }
  const bool write = block == 0;
  int at = before[0];
  if (write || (works && mine == 0 && first >= at && first < at + sum[0]))
#pragma unroll 1
    for (int p = p0; p < p1; ++p) {
      const int n = p0 + 1 == p1 ? sum[0] : Group(g, p).all(g);
      if (write) g.s.tiles_g[p] = at;
      if (mine == 0 && first >= at && first < at + n) out->p = p, out->before = at;
      at += n;
    }
  at = before[1];
  if (works && mine == 1 && first >= at && first < at + sum[1]) {
    int p = at0;
#pragma unroll 1
    for (int b = b0; b < b1; ++b) {
      const int n = own_tiles(b, &p) * g.a.Hkv;
      if (first >= at && first < at + n) out->b = b, out->pb = p, out->before = at;
      at += n;
    }
  }
  __syncthreads();
  if (write) {
    if (tid == 0) *g.s.line = Line{{total[0], total[1]}, {W0, W1}};
    const int G = g.a.Hq / g.a.Hkv;
    int p = at0;
    at = before[1];
#pragma unroll 1
    for (int b = b0; b < b1; ++b) {
      Row r;
      r.n = own_tiles(b, &p);
      r.own = at;
      at += r.n * g.a.Hkv;
      const Group gr(g, p);
      const int L = sched::clamp_len(g.cache_len, b, cap);
      r.span = -1;
      r.pre = r.pre_head = r.entry = 0;
      r.entry_head = r.pad = 0;
      if (shared_of(g, gr, b, L) > 0) {
        const int piece = (b - gr.s0) / (2 * g.seqs);
        r.span = gr.tiles - 1;
        r.pre = g.s.tiles_g[p] + piece * gr.tiles;
        r.pre_head = gr.supers * gr.tiles;
        r.entry = gr.s0 * g.a.Hq + (b - gr.s0) * G;
        r.entry_head = (gr.s1 - gr.s0) * G;
      }
      g.s.rows[b] = r;
    }
  }
}

// One prefix segment: keys [k0, k1) of (group, head, piece).
struct PSegment {
  int p, head, k0, k1;
  int s0, n;                   // the piece's sequences
  bool both;                   // it has rows for both tiles
  int entry;                   // place of its first partial result
  __device__ __forceinline__ int blocks() const { return (k1 - k0 + kKeys - 1) / kKeys; }
  // Does tile t take the segment's key tile j?
  __device__ __forceinline__ bool need(int t, int j) const { return both || (j & 1) == t; }
  // The number of key tiles that tile t takes.
  __device__ __forceinline__ int count(int t) const {
    return both ? blocks() : (blocks() + 1 - t) >> 1;
  }
};

// Places of a piece's rows before those of its pair's segments of other workers.
__device__ __forceinline__ int first_entry(const Plan& g, const Group& p, int head, int piece) {
  const int G = g.a.Hq / g.a.Hkv;
  return p.s0 * g.a.Hq + head * (p.s1 - p.s0) * G + 2 * piece * g.seqs * G;
}

struct PrefixWalk {
  const Plan& g;
  int p, w;
  int at, last, before;
  __device__ __forceinline__ PrefixWalk(const Plan& g_, const SharedStart& s)
      : g(g_), p(s.p), w(s.w), at(s.first), last(s.last), before(s.before) {}
  __device__ __forceinline__ bool next(PSegment& sg) {
    if (at >= last) return false;
#pragma unroll 1
    for (; p < g.groups; ++p) {
      const Group gr(g, p);
      const int all = gr.all(g);
      if (at < before + all) {
        const int pair = (at - before) / gr.tiles;
        const int pair_start = before + pair * gr.tiles;
        const int piece = pair % gr.supers;
        const int g1 = min(gr.tiles, last - pair_start);
        sg.p = p;
        sg.head = pair / gr.supers;
        sg.k0 = static_cast<int>(at - pair_start) * kKeys;
        sg.k1 = min(g1 * kKeys, gr.keys);
        sg.s0 = gr.s0 + piece * 2 * g.seqs;
        sg.n = min(2 * g.seqs, gr.s1 - sg.s0);
        sg.both = sg.n > g.seqs;
        sg.entry = first_entry(g, gr, sg.head, piece) + 2 * w * g.seqs * (g.a.Hq / g.a.Hkv);
        at = pair_start + g1;
        return true;
      }
      before += all;
    }
    return false;
  }
};

// The first segment begins inside a pair, the others with one.
struct OwnWalk {
  const Plan& g;
  int b, p, w, head, g0;
  int left;                    // tiles of the worker's range that are still to come
  int L, from, n;              // of sequence b: length, first own token, tiles of a head
  __device__ __forceinline__ OwnWalk(const Plan& g_, const SharedStart& s)
      : g(g_), b(s.b), p(s.pb), w(s.w), left(s.last - s.first) {
    if (left <= 0) return;
    sequence();
    const int x = s.first - s.before;
    head = x / n;                                // find_start has found the sequence that holds it
    g0 = x - head * n;
  }
  __device__ __forceinline__ void sequence() {
#pragma unroll 1
    while (p + 1 < g.groups && g.start[p + 1] <= b) ++p;
    const Group gr(g, p);
    L = sched::clamp_len(g.cache_len, b, cap_of(g.a));
    from = shared_of(g, gr, b, L);
    n = sched::granules<kKeys>(L - from);
    head = 0;
  }
  __device__ __forceinline__ bool next(Segment& sg) {
    if (left <= 0) return false;
    while (head >= g.a.Hkv || n == 0) {
      if (++b >= g.a.B) return false;
      sequence();
    }
    const int g1 = min(n, g0 + left);
    sg.b = b;
    sg.head = head;
    sg.len = L;
    sg.k0 = from + g0 * kKeys;
    sg.k1 = min(from + g1 * kKeys, L);
    sg.whole = from == 0 && g0 == 0 && g1 == n;
    sg.slot = b * g.a.Hkv + head + w;
    left -= g1 - g0;
    g0 = 0;
    ++head;
    return true;
  }
};

template <int D>
__device__ __forceinline__ void prefix_segments(const CUtensorMap& mk, const CUtensorMap& mv,
                                                const CUtensorMap& mr, const Plan& g,
                                                uint8_t* base, PBars* bars, uint32_t tb,
                                                PrefixWalk walk) {
  using C = PC<D>;
  const PagedArgs& a = g.a;
  uint8_t* sQ = base;                            // [2][TILE]
  uint8_t* sK = sQ + 2 * C::TILE;                // [NK][TILE]
  uint8_t* sV = sK + C::NK * C::TILE;            // [NV][TILE]
  volatile int* abort_flag = &bars->abort;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int G = a.Hq / a.Hkv;
  PSegment sg;

  if (warp == 0 || warp == 2) {
    // ------------------------------------------------------------ TMA producers
    const bool keys = warp == 0;
    const CUtensorMap* map = keys ? &mk : &mv;
    uint64_t* full = keys ? bars->k_full : bars->v_full;
    uint64_t* empty = keys ? bars->k_empty : bars->v_empty;
    const int shift = a.page_shift;
    const int rows = min(kBox, 1 << shift), boxes = kKeys / rows;
    const uint32_t bits = (1u << (rows / 16)) - 1u;
    const int stages = keys ? C::NK : C::NV;
    bool ok = true;
    int n = 0, ns = 0, st = 0;
    uint32_t round = 0;                          // of the stages
    while (ok && walk.next(sg)) {
      if (!keys) {   // the queries with the values, which are needed later than the first keys
        if (ns > 0) {
          ok = mbar_wait_warp(&bars->q_empty, (ns - 1) & 1, abort_flag, a.err, a.wait_ns);
          if (!ok) break;
        }
        if (lane == 0) {
          const uint32_t box = static_cast<uint32_t>(g.seqs) * G * 128;
          mbar_arrive_expect_tx(&bars->q_full, 2 * C::NSUB * box);
#pragma unroll 1
          for (int t = 0; t < 2; ++t)
            for (int s = 0; s < C::NSUB; ++s)
              tma_load_4d(sQ + t * C::TILE + s * kSub, &mr, &bars->q_full, 64 * s, 0, sg.head,
                          sg.s0 + (sg.both ? t * g.seqs : 0));
        }
      }
      // The table row of the group's first sequence that has all of the shared tokens.
      const Group gr(g, sg.p);
      int rep = -1;
#pragma unroll 1
      for (int b = gr.s0; rep < 0 && b < gr.s1; b += 32) {
        const bool has = b + lane < gr.s1 &&
                         sched::clamp_len(g.cache_len, b + lane, cap_of(a)) >= gr.len;
        const uint32_t hit = __ballot_sync(0xffffffffu, has);
        if (hit) rep = b + __ffs(hit) - 1;
      }
      const int32_t* row = a.table + max(rep, 0) * a.table_stride;
      for (int k0 = sg.k0; k0 < sg.k1; k0 += kKeys, ++n) {
        const int x = k0 + lane * rows;
        int p = -1;
        if (lane < boxes && x < sg.k1 && rep >= 0) p = row[x >> shift];
        const bool in = p >= 0 && p < a.num_pages;
        const uint32_t pages = __ballot_sync(0xffffffffu, in);
        if (round > 0) {
          ok = mbar_wait_warp(&empty[st], (round - 1) & 1, abort_flag, a.err, a.wait_ns);
          if (!ok) break;
        }
        if (lane == 0) {
          if (keys) {
            uint32_t seen = 0;
#pragma unroll 1
            for (int i = 0; i < boxes; ++i)
              if (pages >> i & 1u) seen |= bits << (i * (rows / 16));
            bars->seen[n % kSeen] = seen;
          }
          mbar_arrive_expect_tx(&full[st], static_cast<uint32_t>(__popc(pages)) * rows * D * 2);
        }
        __syncwarp();
        if (in) {
          uint8_t* dst = (keys ? sK : sV) + st * C::TILE + lane * rows * 128;
          const int y = x & ((1 << shift) - 1);
#pragma unroll
          for (int s = 0; s < C::NSUB; ++s)
            tma_load_4d(dst + s * kSub, map, &full[st], 64 * s, y, sg.head, p);
        }
        if (++st == stages) st = 0, ++round;
      }
      ++ns;
    }
  } else if (warp == 1 || warp == 3) {
    // ------------------------------------------------------------ MMA issuers, one a tile
    // Both walk every stage (a stage is free when both have released it).  In the order of one
    // thread's MMAs the scores of the tile's next key tile follow the product that reads its P.
    if (lane == 0) {
      const int t = warp == 1 ? 0 : 1;
      constexpr uint32_t idS = idesc_bf16(128, 128, false, false);
      constexpr uint32_t idO = idesc_bf16(128, D, false, true);
      const uint64_t dQ = sw128_desc(smem_u32(sQ + t * C::TILE), 16, 1024);
      const uint64_t dK0 = sw128_desc(smem_u32(sK), 16, 1024);
      const uint64_t dV0 = sw128_desc(smem_u32(sV), kSub, 1024);
      constexpr uint64_t kTileD = C::TILE >> 4;
      const uint32_t tS = tb + t * 128, tO = tb + 256 + t * 128;
      bool ok = true;
      int n = 0, ns = 0, npv = 0, nout = 0;
      auto scores = [&](int m) {         // of the m-th key tile
        const uint64_t dK = dK0 + static_cast<uint64_t>(m % C::NK) * kTileD;
#pragma unroll
        for (int q = 0; q < C::NSUB; ++q) {
          uint64_t da[4], db[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const uint64_t off = static_cast<uint64_t>((q * kSub + k * 32) >> 4);
            da[k] = dQ + off;
            db[k] = dK + off;
          }
          mma_ss_x4(tS, da, db, idS, q > 0 ? 1u : 0u);
        }
        mma_commit(&bars->s_full[t]);
      };
      auto keys_in = [&](int m) {
        ok = mbar_wait(&bars->k_full[m % C::NK], (m / C::NK) & 1, abort_flag, a.err, a.wait_ns);
        tc_fence_after();
        return ok;
      };
      while (ok && walk.next(sg)) {
        const int blocks = sg.blocks(), mine = sg.count(t);
        ok = mbar_wait(&bars->q_full, ns & 1, abort_flag, a.err, a.wait_ns);
        if (!ok || !keys_in(n)) break;
        if (sg.need(t, 0)) scores(n);
        mma_commit(&bars->k_empty[n % C::NK]);
        if (blocks == 1) mma_commit(&bars->q_empty);
        int done = 0;
        for (int j = 0; j < blocks; ++j, ++n) {
          ok = mbar_wait(&bars->v_full[n % C::NV], (n / C::NV) & 1, abort_flag, a.err, a.wait_ns);
          // the next keys too, so that their scores are issued right behind this product
          if (!ok || (j + 1 < blocks && !keys_in(n + 1))) break;
          if (sg.need(t, j)) {
            ok = mbar_wait(&bars->p_full[t], npv & 1, abort_flag, a.err, a.wait_ns);
            // the previous segment's O has been read
            if (ok && done == 0 && nout > 0)
              ok = mbar_wait(&bars->o_empty[t], (nout - 1) & 1, abort_flag, a.err, a.wait_ns);
            if (!ok) break;
            tc_fence_after();
            const uint64_t dV = dV0 + static_cast<uint64_t>(n % C::NV) * kTileD;
#pragma unroll
            for (int q = 0; q < 2; ++q) {
              uint32_t ta[4];
              uint64_t db[4];
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                ta[k] = tS + 8 * (4 * q + k);
                db[k] = dV + static_cast<uint64_t>((2048 * (4 * q + k)) >> 4);
              }
              mma_ts_x4(tO, ta, db, idO, (done > 0 || q > 0) ? 1u : 0u);
            }
            ++npv;
            if (++done == mine) mma_commit(&bars->o_done[t]);
          }
          mma_commit(&bars->v_empty[n % C::NV]);
          if (j + 1 < blocks) {
            if (sg.need(t, j + 1)) scores(n + 1);
            mma_commit(&bars->k_empty[(n + 1) % C::NK]);
            if (j + 2 == blocks) mma_commit(&bars->q_empty);
          }
        }
        if (mine > 0) ++nout;
        ++ns;
      }
      // Every MMA issued by either thread has completed before tensor memory is used again.
      mma_commit(&bars->drain);
      mbar_wait(&bars->drain, 0, &bars->never, nullptr, a.wait_ns);
    }
  } else if (warp >= 4) {
    // ------------------------------------------------------------ softmax warps
    // Warp 4 + q + 4 h owns rows 32 q + 16 h + [0, 16) of both tiles: thread t has rows
    // A = 32 q + 16 h + t / 4 and B = A + 8, keys 8 c + 2 (t % 4) + {0, 1}.
    const int q4 = warp & 3, hh = (warp - 4) >> 2, t4 = lane & 3;
    const int rA = 32 * q4 + 16 * hh + (lane >> 2), rB = rA + 8;
    const uint32_t lane_base = tb + (static_cast<uint32_t>(32 * q4 + 16 * hh) << 16);
    const uint64_t c2 = f2_pack(a.c, a.c);
    int n = 0, n_s[2] = {0, 0}, n_out[2] = {0, 0};
    bool ok = true;
    while (ok && walk.next(sg)) {
      const int blocks = sg.blocks();
      float m_run[2][2] = {{-INFINITY, -INFINITY}, {-INFINITY, -INFINITY}};
      float l_part[2][2] = {{0.f, 0.f}, {0.f, 0.f}};
      // One copy of the code for both tiles (state [0] is the current one's): it has to share the
      // instruction caches with the continuations'.
#pragma unroll 1
      for (int jt = 0; jt < 2 * blocks; ++jt) {
        const int j = jt >> 1, t = jt & 1;
        if (sg.need(t, j)) {
          ok = mbar_wait_warp(&bars->s_full[t], n_s[0] & 1, abort_flag, a.err, a.wait_ns);
          if (!ok) break;
          tc_fence_after();
          uint32_t v[64];
          tmem_ld_16x256b_x16_wait(lane_base + t * 128, v);
          float sv[64];
#pragma unroll
          for (int i = 0; i < 64; ++i) sv[i] = __uint_as_float(v[i]);
          const uint32_t seen = bars->seen[n % kSeen];
          const int lim = min(sg.k1 - (sg.k0 + j * kKeys), kKeys);
          const bool edge = lim < kKeys || seen != 0xffu;
          if (edge) {
#pragma unroll
            for (int cc = 0; cc < 16; ++cc) {
              // the limit is a multiple of 16, as the pages are
              if (16 * (cc >> 1) >= lim || !((seen >> (cc >> 1)) & 1u))
                sv[4 * cc] = sv[4 * cc + 1] = sv[4 * cc + 2] = sv[4 * cc + 3] = -INFINITY;
            }
          }
          float ma0 = fmaxf(sv[0], sv[1]), ma1 = fmaxf(sv[4], sv[5]);
          float mb0 = fmaxf(sv[2], sv[3]), mb1 = fmaxf(sv[6], sv[7]);
#pragma unroll
          for (int cc = 2; cc < 16; cc += 2) {
            ma0 = fmax3(ma0, sv[4 * cc], sv[4 * cc + 1]);
            mb0 = fmax3(mb0, sv[4 * cc + 2], sv[4 * cc + 3]);
            ma1 = fmax3(ma1, sv[4 * cc + 4], sv[4 * cc + 5]);
            mb1 = fmax3(mb1, sv[4 * cc + 6], sv[4 * cc + 7]);
          }
          float mA = fmaxf(ma0, ma1), mB = fmaxf(mb0, mb1);
          mA = fmaxf(mA, __shfl_xor_sync(0xffffffffu, mA, 1));
          mB = fmaxf(mB, __shfl_xor_sync(0xffffffffu, mB, 1));
          mA = fmaxf(mA, __shfl_xor_sync(0xffffffffu, mA, 2));
          mB = fmaxf(mB, __shfl_xor_sync(0xffffffffu, mB, 2));
          mA *= a.c;
          mB *= a.c;
          const float oldA = m_run[0][0], oldB = m_run[0][1];
          const float newA = mA > oldA + kRescaleThreshold ? mA : oldA;
          const float newB = mB > oldB + kRescaleThreshold ? mB : oldB;
          const bool chA = newA != oldA, chB = newB != oldB;
          const float alphaA = chA ? ex2(oldA - newA) : 1.f;   // old = -inf gives 0
          const float alphaB = chB ? ex2(oldB - newB) : 1.f;
          const float useA = newA == -INFINITY ? 0.f : newA;
          const float useB = newB == -INFINITY ? 0.f : newB;
          const uint64_t nA = f2_pack(-useA, -useA), nB = f2_pack(-useB, -useB);
          uint64_t accA = f2_pack(0.f, 0.f), accB = accA;
          uint32_t pk[32];
#pragma unroll
          for (int cc = 0; cc < 16; ++cc) {
            const float2 xa = f2_unpack(ffma2(f2_pack(sv[4 * cc], sv[4 * cc + 1]), c2, nA));
            const float2 xb = f2_unpack(ffma2(f2_pack(sv[4 * cc + 2], sv[4 * cc + 3]), c2, nB));
            const float pa0 = ex2(xa.x), pa1 = ex2(xa.y);
            const float pb0 = ex2(xb.x), pb1 = ex2(xb.y);
            accA = fadd2(accA, f2_pack(pa0, pa1));
            accB = fadd2(accB, f2_pack(pb0, pb1));
            pk[2 * cc] = pack_bf16x2(pa0, pa1);
            pk[2 * cc + 1] = pack_bf16x2(pb0, pb1);
          }
          tmem_st_16x128b_x16(lane_base + t * 128, pk);
          const float2 sa = f2_unpack(accA), sb = f2_unpack(accB);
          l_part[0][0] = l_part[0][0] * alphaA + (sa.x + sa.y);
          l_part[0][1] = l_part[0][1] * alphaB + (sb.x + sb.y);
          m_run[0][0] = newA;
          m_run[0][1] = newB;
          // Rescale the running O; the products issued before the scores just read are done.
          if (j > (sg.both ? 0 : t) && __any_sync(0xffffffffu, chA || chB)) {
#pragma unroll
            for (int half = 0; half < D / 64; ++half) {
              uint32_t o[32];
              const uint32_t oaddr = lane_base + 256 + t * 128 + 64 * half;
              tmem_ld_16x256b_x8_wait(oaddr, o);
#pragma unroll
              for (int i = 0; i < 32; ++i)
                o[i] = __float_as_uint(__uint_as_float(o[i]) * ((i & 2) ? alphaB : alphaA));
              tmem_st_16x256b_x8(oaddr, o);
            }
          }
          if (edge && (t == 0 || !sg.both)) {
            // Hidden rows of V: zero, so that 0 x (anything) stays 0.  The stage is this tile's once
            // its load has completed.
            ok = mbar_wait_warp(&bars->v_full[n % C::NV], (n / C::NV) & 1, abort_flag, a.err,
                                a.wait_ns);
            if (!ok) break;
            const int i = tid - 128, r = i & 127;
            if (r >= lim || !((seen >> (r >> 4)) & 1u)) {
              uint8_t* vt = sV + (n % C::NV) * C::TILE + r * 128;
#pragma unroll
              for (int ch = 0; ch < 4 * C::NSUB; ++ch) {
                // 16-byte pieces of the row, every lane from another one on (banks)
                const int at = (i >> 7) * 4 * C::NSUB + ((ch + lane) & (4 * C::NSUB - 1));
                *reinterpret_cast<uint4*>(vt + (at >> 3) * kSub + (at & 7) * 16) =
                    make_uint4(0, 0, 0, 0);
              }
            }
            fence_proxy_async_smem();
          }
          tmem_wait_st();
          tc_fence_before();
          mbar_arrive(&bars->p_full[t]);
          ++n_s[0];
        }
        n += t;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float m = m_run[0][i], l = l_part[0][i];
          m_run[0][i] = m_run[1][i], l_part[0][i] = l_part[1][i];
          m_run[1][i] = m, l_part[1][i] = l;
        }
        const int s = n_s[0];
        n_s[0] = n_s[1];
        n_s[1] = s;
      }
      if (!ok) break;
      // ---- the segment's partial results; tiles with the same rows are joined first
      const bool two = sg.count(1) > 0, join = !sg.both && two;
      ok = mbar_wait_warp(&bars->o_done[0], n_out[0] & 1, abort_flag, a.err, a.wait_ns);
      ++n_out[0];
      if (ok && two) {
        ok = mbar_wait_warp(&bars->o_done[1], n_out[1] & 1, abort_flag, a.err, a.wait_ns);
        ++n_out[1];
      }
      if (!ok) break;
      tc_fence_after();
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          l_part[t][i] += __shfl_xor_sync(0xffffffffu, l_part[t][i], 1);
          l_part[t][i] += __shfl_xor_sync(0xffffffffu, l_part[t][i], 2);
        }
      float w[2][2] = {{1.f, 1.f}, {0.f, 0.f}};    // of the tiles' rows A and B, where they are joined
      if (join) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float M = fmaxf(m_run[0][i], m_run[1][i]), use = M == -INFINITY ? 0.f : M;
          w[0][i] = ex2(m_run[0][i] - use);        // -inf gives 0
          w[1][i] = ex2(m_run[1][i] - use);
          m_run[0][i] = M;
          l_part[0][i] = l_part[0][i] * w[0][i] + l_part[1][i] * w[1][i];
        }
      }
      // One copy of the code for the tiles and their halves, as above.
#pragma unroll 1
      for (int th = 0; th < (sg.both ? 2 : 1) * (D / 64); ++th) {
        const int t = th / (D / 64), half = th % (D / 64);
        // Rows of the tile, and the place of its first; group starts that are not ascending may
        // lead past the end, where nothing is written.
        const int rows = (sg.both ? (t == 0 ? g.seqs : sg.n - g.seqs) : sg.n) * G;
        const int e0 = sg.entry + t * g.seqs * G;
        const bool wA = rA < rows && e0 + rA < g.s.entries, wB = rB < rows && e0 + rB < g.s.entries;
        float* outA = g.s.part + (e0 + rA) * D + 64 * half;
        float* outB = g.s.part + (e0 + rB) * D + 64 * half;
        uint32_t ov[32];
        tmem_ld_16x256b_x8_wait(lane_base + 256 + t * 128 + 64 * half, ov);
        if (join) {
          uint32_t o1[32];
          tmem_ld_16x256b_x8_wait(lane_base + 384 + 64 * half, o1);
#pragma unroll
          for (int i = 0; i < 32; ++i)
            ov[i] = __float_as_uint(__uint_as_float(ov[i]) * w[0][(i >> 1) & 1] +
                                    __uint_as_float(o1[i]) * w[1][(i >> 1) & 1]);
        }
        // Neighbouring threads of a row exchange halves of two column groups: four columns each.
        const int odd = t4 & 1;
#pragma unroll
        for (int cc = 0; cc < 8; cc += 2) {
          const int col = 8 * (cc + odd) + 4 * (t4 >> 1);
#pragma unroll
          for (int i = 0; i < 2; ++i) {        // row A, row B
            const uint32_t* u = ov + 4 * cc + 2 * i;
            const uint32_t x = __shfl_xor_sync(0xffffffffu, odd ? u[0] : u[4], 1);
            const uint32_t y = __shfl_xor_sync(0xffffffffu, odd ? u[1] : u[5], 1);
            const uint4 q = odd ? make_uint4(x, y, u[4], u[5]) : make_uint4(u[0], u[1], x, y);
            if (i ? wB : wA) *reinterpret_cast<uint4*>((i ? outB : outA) + col) = q;
          }
        }
        if (t4 == 0 && half == 0) {
          if (wA) g.s.stats[e0 + rA] = make_float2(t ? m_run[1][0] : m_run[0][0], t ? l_part[1][0] : l_part[0][0]);
          if (wB) g.s.stats[e0 + rB] = make_float2(t ? m_run[1][1] : m_run[0][1], t ? l_part[1][1] : l_part[0][1]);
        }
      }
      tc_fence_before();
      mbar_arrive(&bars->o_empty[0]);
      if (two) mbar_arrive(&bars->o_empty[1]);
    }
  }
}

static_assert(TC<64>::SMEM + sizeof(Lists) + 600 <= 227 * 1024 &&
                  TC<128>::SMEM + sizeof(Lists) + 600 <= 227 * 1024, "shared memory");

template <int D, int GP>
__global__ void __launch_bounds__(kThreads, 1)
decode_shared_kernel(const __grid_constant__ CUtensorMap mk, const __grid_constant__ CUtensorMap mv,
                     const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mr,
                     const __grid_constant__ SharedArgs g) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  __shared__ PBars pb;
  const Smem<D> sh(base);
  Bars* db = sh.bars;                            // of the continuations
  __shared__ SharedStart start;
  __shared__ Sums scan[kThreads / 32];
  __shared__ Lists lists;
  const int tid = threadIdx.x, warp = tid >> 5;

  if (tid == 0) {
    mbar_init(&pb.q_full, 1);
    mbar_init(&pb.q_empty, 2);
    for (int s = 0; s < 4; ++s) {
      mbar_init(&pb.k_full[s], 1);
      mbar_init(&pb.k_empty[s], 2);
      mbar_init(&pb.v_full[s], 1);
      mbar_init(&pb.v_empty[s], 2);
    }
    for (int t = 0; t < 2; ++t) {
      mbar_init(&pb.s_full[t], 1);
      mbar_init(&pb.p_full[t], 256);
      mbar_init(&pb.o_done[t], 1);
      mbar_init(&pb.o_empty[t], 256);
    }
    mbar_init(&pb.drain, 2);
    pb.abort = 0;
    pb.never = 0;
    init_bars<D>(db);
    tma_prefetch_desc(&mk);
    tma_prefetch_desc(&mv);
    tma_prefetch_desc(&mq);
    tma_prefetch_desc(&mr);
  }
  if (warp == 2) {
    tmem_alloc(&pb.tmem_base, 512);
    tmem_relinquish();
  }
  griddep_wait();
  griddep_launch_dependents();
  const Plan plan(g, &lists);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  find_start(&start, scan, plan);
  const uint32_t tb = pb.tmem_base;
  if (start.first < start.last) {
    if (start.mine == 0)
      prefix_segments<D>(mk, mv, mr, plan, base, &pb, tb, PrefixWalk(plan, start));
    else
      segments<D, GP>(mk, mv, mq, g.a, sh, tb, OwnWalk(plan, start));
  }

  tc_fence_before();
  __syncthreads();
  if ((pb.abort || db->abort) && tid == 0) {
    // Let any copy still in flight land before the CTA's shared memory is released.
    const uint64_t t0 = globaltimer();
    while (globaltimer() - t0 < 1000000ull) {
    }
  }
  __syncthreads();
  if (warp == 2) {
    tc_fence_after();
    tmem_dealloc(tb, 512);
  }
}

// Joins a row's partial results; o = 0, lse = -inf for an empty sequence.  W warps (1, 2 or 4) per
// (sequence, query head), each with every W-th part.
template <int D, int W>
__global__ void __launch_bounds__(256, 4) decode_shared_combine_kernel(
    const __grid_constant__ SharedArgs g) {
  constexpr int PS = TC<D>::PSTRIDE, PER = D / 32;
  __shared__ float red[8][D + 2];                // a warp's columns, maximum and sum
  griddep_wait();
  griddep_launch_dependents();
  const PagedArgs& a = g.a;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, sub = warp % W, G = a.Hq / a.Hkv;
  const int row = blockIdx.x * (8 / W) + warp / W;
  const bool live = row < a.B * a.Hq;
  const int b = live ? static_cast<int>(row / a.Hq) : 0, hq = live ? static_cast<int>(row % a.Hq) : 0;
  const int head = hq / G, h = hq % G;
  const Line line = *g.line;
  const Row r = g.rows[b];
  int own = 0, pre = 0, step = 0;                // parts of the continuation, of the prefix
  const float* own0 = nullptr;                   // the first ones
  int pre0 = 0;
  if (r.n > 0 && line.workers[1] > 0) {
    const int first = r.own + head * r.n;
    const int w0 = owner(first, line.total[1], line.workers[1]);
    own = owner(first + r.n - 1, line.total[1], line.workers[1]) - w0 + 1;
    own0 = a.part + ((b * a.Hkv + head + w0) * G + h) * PS;
  }
  if (r.span >= 0 && line.workers[0] > 0) {
    const int first = r.pre + head * r.pre_head;
    const int w0 = owner(first, line.total[0], line.workers[0]);
    pre = owner(first + r.span, line.total[0], line.workers[0]) - w0 + 1;
    step = 2 * g.seqs * G;
    pre0 = r.entry + head * r.entry_head + h + w0 * step;
    pre = min(pre, (g.entries - 1 - pre0) / step + 1);
  }
  // A continuation that is all of its rows' keys and one CTA's is finished; W > 1: the block goes on
  // to its barrier.
  const bool todo = live && !(r.span < 0 && own == 1);
  const int parts = todo ? pre + own : 0;
  auto o_at = [&](int i) {
    return i < pre ? g.part + (pre0 + i * step) * D
                   : own0 + (i - pre) * G * PS;
  };
  auto stats_at = [&](int i) {
    return i < pre ? g.stats + (pre0 + i * step)
                   : reinterpret_cast<const float2*>(own0 + (i - pre) * G * PS + D);
  };
  float acc[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) acc[i] = 0.f;
  float M = -INFINITY, lsum = 0.f;
  for (int base = sub; base < parts; base += 32 * W) {
    const int mine = base + lane * W;
    const int cnt = min(32, (parts - base + W - 1) / W);
    // Eight parts' loads in flight, the first ones beside their statistics'; those past the last repeat
    // it with weight 0.
    float v[8][PER];
    auto load = [&](int j0) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float* pj = o_at(base + min(j0 + j, cnt - 1) * W) + lane * PER;
        if constexpr (PER == 4) {
          const float4 x = *reinterpret_cast<const float4*>(pj);
          v[j][0] = x.x, v[j][1] = x.y, v[j][2] = x.z, v[j][3] = x.w;
        } else {
          const float2 x = *reinterpret_cast<const float2*>(pj);
          v[j][0] = x.x, v[j][1] = x.y;
        }
      }
    };
    const float2 ml = *stats_at(mine < parts ? mine : base);
    load(0);
    const float m = mine < parts ? ml.x : -INFINITY, l = mine < parts ? ml.y : 0.f;
    const float mb = fmaxf(M, warp_max(m));
    const float use = mb == -INFINITY ? 0.f : mb;
    const float keep = ex2(M - use);             // M = -inf gives 0
    const float wt = ex2(m - use);               // a part without a visible key weighs 0
    M = mb;
    lsum = lsum * keep + l * wt;                 // without a key l is 0, of a NaN query NaN
#pragma unroll
    for (int i = 0; i < PER; ++i) acc[i] *= keep;
    for (int j0 = 0; j0 < cnt; j0 += 8) {
      if (j0 > 0) load(j0);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float wj = __shfl_sync(0xffffffffu, wt, (j0 + j) & 31);
        if (j0 + j >= cnt) break;
#pragma unroll
        for (int i = 0; i < PER; ++i) acc[i] = fmaf(wj, v[j][i], acc[i]);
      }
    }
  }
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) lsum += __shfl_xor_sync(0xffffffffu, lsum, off);
  if constexpr (W > 1) {
#pragma unroll
    for (int i = 0; i < PER; ++i) red[warp][lane * PER + i] = acc[i];
    if (lane == 0) {
      red[warp][D] = M;
      red[warp][D + 1] = lsum;
    }
    __syncthreads();
    if (sub > 0) return;
    float mw[W];
    M = -INFINITY;
#pragma unroll
    for (int w = 0; w < W; ++w) M = fmaxf(M, mw[w] = red[warp + w][D]);
    const float use = M == -INFINITY ? 0.f : M;
    lsum = 0.f;
#pragma unroll
    for (int i = 0; i < PER; ++i) acc[i] = 0.f;
#pragma unroll
    for (int w = 0; w < W; ++w) {
      const float wt = ex2(mw[w] - use);
      lsum += red[warp + w][D + 1] * wt;
#pragma unroll
      for (int i = 0; i < PER; ++i) acc[i] = fmaf(red[warp + w][lane * PER + i], wt, acc[i]);
    }
  }
  if (!todo) return;
  const float inv = lsum == 0.f ? 0.f : 1.f / lsum;   // a NaN sum stays one
  __nv_bfloat16* orow = a.o + static_cast<size_t>(row) * D + lane * PER;
#pragma unroll
  for (int i = 0; i < PER; i += 2)
    *reinterpret_cast<uint32_t*>(orow + i) = pack_bf16x2(acc[i] * inv, acc[i + 1] * inv);
  if (lane == 0) a.lse[row] = lsum == 0.f ? -INFINITY : (M + __log2f(lsum)) * kLn2;
}

template <int D, int W>
cudaError_t launch_combine(const SharedArgs& g, long long rows, cudaStream_t s) {
  constexpr int kEach = 8 / W;
  return launch_dependent(decode_shared_combine_kernel<D, W>,
                          dim3(static_cast<unsigned>((rows + kEach - 1) / kEach)), dim3(256), 0, s,
                          g);
}

template <int D, int GP>
cudaError_t launch_g(const CUtensorMap& mk, const CUtensorMap& mv, const CUtensorMap& mq,
                     const CUtensorMap& mr, const SharedArgs& g, int workers, cudaStream_t s) {
  static std::atomic<bool> attr_set[64];  // per device; a race repeats the same call
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev < 0 || dev >= 64 || !attr_set[dev].load()) {
    cudaError_t e = cudaFuncSetAttribute(decode_shared_kernel<D, GP>,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize, TC<D>::SMEM);
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < 64) attr_set[dev].store(true);
  }
  // An ordinary launch: placed on the SMs while the kernel before still runs, some CTAs took nearly
  // twice as long as the rest to their end (16 groups of 4 sequences, 2048 + 128 tokens: 66 us, 50 with
  // the ordinary launch; the cause is not known).
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(workers);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = TC<D>::SMEM;
  cfg.stream = s;
  cudaError_t e = cudaLaunchKernelEx(&cfg, decode_shared_kernel<D, GP>, mk, mv, mq, mr, g);
  if (e != cudaSuccess) return e;
  // As many warps a row as are resident at once (four blocks an SM): 64 sequences of 32 heads, 8192 +
  // 512 tokens, with two waves of blocks 1.5 us more.
  const long long rows = static_cast<long long>(g.a.B) * g.a.Hq, most = 32ll * sm_count();
  if (4 * rows <= most) return launch_combine<D, 4>(g, rows, s);
  if (2 * rows <= most) return launch_combine<D, 2>(g, rows, s);
  return launch_combine<D, 1>(g, rows, s);
}

template <int D>
cudaError_t launch_d(const void* q, const void* k, const void* v, long long page_stride,
                     const SharedArgs& g, int workers, cudaStream_t s) {
  CUtensorMap mk, mv, mq, mr;
  const PagedArgs& a = g.a;
  const int page = 1 << a.page_shift, rows = page < kBox ? page : kBox, G = a.Hq / a.Hkv;
  // The rows of a prefix tile: G heads of `seqs` sequences, from [B, Hkv, G, d].
  if (!make_page_map(&mk, k, a.num_pages, a.Hkv, page, D, page_stride, rows) ||
      !make_page_map(&mv, v, a.num_pages, a.Hkv, page, D, page_stride, rows) ||
      !make_head_map_rows(&mq, q, 1, a.B * a.Hq, D, kN) ||
      !make_query_map(&mr, q, a.B, a.Hkv, G, D, g.seqs))
    return cudaErrorInvalidValue;
  if (G > 8) return launch_g<D, 16>(mk, mv, mq, mr, g, workers, s);
  if (G > 4) return launch_g<D, 8>(mk, mv, mq, mr, g, workers, s);
  if (G > 2) return launch_g<D, 4>(mk, mv, mq, mr, g, workers, s);
  if (G > 1) return launch_g<D, 2>(mk, mv, mq, mr, g, workers, s);
  return launch_g<D, 1>(mk, mv, mq, mr, g, workers, s);
}

// Places for the prefixes' partial results: one a row, and a piece's rows for every worker that begins
// inside a pair.
int prefix_entries(int B, int Hq, int G) {
  return B * Hq + 2 * sm_count() * (kRows / G) * G;
}
int own_entries(int B, int Hkv, int G) {
  return (B * Hkv + sm_count()) * G;
}

// Is there so little to read that sharing it costs more than it saves?  Apart the sequences have
// `tiles` tiles (by the width of the table; the lengths are on the device), some 1 us an SM each; the
// two kinds of CTAs and the join add 3 to 5 us, and what they save grows with the sequences a group.
// Measured (d = 64 and 128, 1 to 16 heads a group, one key/value head to eight; tiles an SM at which
// both take as long): groups of 2 sequences 25 to 30, of 4 14, of 8 10, of 16 and more 5 to 7.  Four
// sequences of 700 tokens: 11.4 us shared, 8.9 apart; 32 of 1084 tokens, d = 128, 8 key/value heads,
// one group (15 tiles an SM): 16.0 and 23.5.
bool decode_apart(long long tiles, int B, int groups) {
  return tiles * B <= (4ll * B + 40ll * groups) * sm_count();
}

}  // namespace

size_t decode_shared_bytes(int B, int Hq, int Hkv, int d) {
  const int G = Hq / Hkv;
  const size_t entry = (d + 4) * sizeof(float);
  const size_t shared =
      round_up(prefix_entries(B, Hq, G) * (d * sizeof(float) + sizeof(float2)), 256) +
      round_up(own_entries(B, Hkv, G) * entry, 256) + B * (sizeof(Row) + sizeof(int)) +
      sizeof(Line);
  const size_t apart = decode_paged_part_bytes(G, d) +
                       (static_cast<size_t>(B) + 1) * sizeof(long long);
  return shared > apart ? shared : apart;
}

cudaError_t launch_decode_shared(const void* q, const void* k, const void* v,
                                 long long page_stride, const int32_t* table,
                                 long long table_stride, int max_pages, int page_shift,
                                 int num_pages, const int32_t* cache_len, const int32_t* start,
                                 const int32_t* shared_len, int groups, void* o, float* lse, int B,
                                 int Hq, int Hkv, int d, float scale, void* workspace, int* err,
                                 unsigned long long wait_ns, cudaStream_t s) {
  const long long most = (static_cast<long long>(max_pages) << page_shift) + kKeys - 1;
  const long long tiles = static_cast<long long>(B) * Hkv * (most / kKeys);
  if (decode_apart(tiles, B, groups))
    return launch_decode_paged(q, k, v, page_stride, table, table_stride, max_pages, page_shift,
                               num_pages, cache_len, o, lse, B, Hq, Hkv, d, scale, workspace, err,
                               wait_ns, s);
  const int G = Hq / Hkv;
  const size_t entry = (d + 4) * sizeof(float);
  char* at = static_cast<char*>(workspace);
  SharedArgs g{};
  g.entries = prefix_entries(B, Hq, G);
  g.part = reinterpret_cast<float*>(at);
  g.stats = reinterpret_cast<float2*>(g.part + g.entries * d);
  at += round_up(g.entries * (d * sizeof(float) + sizeof(float2)), 256);
  g.a = PagedArgs{table, table_stride, max_pages, page_shift, num_pages, cache_len, B, Hq, Hkv,
                  scale * kLog2e, static_cast<__nv_bfloat16*>(o), lse,
                  reinterpret_cast<float*>(at), nullptr, err, wait_ns};
  at += round_up(own_entries(B, Hkv, G) * entry, 256);
  g.rows = reinterpret_cast<Row*>(at);
  g.line = reinterpret_cast<Line*>(g.rows + B);
  g.tiles_g = reinterpret_cast<int*>(g.line + 1);
  g.start = start;
  g.len = shared_len;
  g.groups = groups;
  g.seqs = kRows / G;
  const int workers = sm_count();                // there may be more tiles
  return d == 64 ? launch_d<64>(q, k, v, page_stride, g, workers, s)
                 : launch_d<128>(q, k, v, page_stride, g, workers, s);
}

}  // namespace fa
