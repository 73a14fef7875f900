// prefix.cu — decode attention of a batch whose sequences share prefixes.
//
// Sequences of a group hold the same pages for their first P blocks.  With the queries of all
// its sequences as rows of one matrix, the prefix is read once for the group:
//   S = Q K^T * scale,  m = rowmax S,  p = 2^(S - m),  l = rowsum p,  O = p V
// (base 2: scale carries log2 e), per row over a range of blocks; what each sequence has of
// its own behind the prefix gives parts of the same form, and the parts (m_i, l_i, O_i) of a
// row join as
//   M = max m_i,  out = sum O_i 2^(m_i - M) / sum l_i 2^(m_i - M).
// Three launches:
//   plan     one CTA: members of each group (sequences that hold the whole prefix; a group
//            of one shares nothing), row tiles, and each CTA's first block.
//   attend   one persistent CTA an SM over equal shares of all blocks.
//   combine  a warp for 8 rows and 16 channels.
// Rows of the tensor-core steps (M = 128) are the queries of a group, as the G <= 8 queries of one
// sequence fill an eighth of the smallest tile and every sequence would read the prefix anew.
//
// What bounds it.  64 sequences of 4 queries a K/V head (8) behind 32K tokens, 270 MB: 90 us, of which
// plan 3, attend 77, combine 6.  Where two tiles of rows share their blocks the tensor cores do: a
// block is 24 products of K = 16 a tile (8 for S, 16 for P in two parts), 2100 cycles where they
// alone would take 1580 (S reads Q and K from shared memory at its full rate, beside which tiles
// land); behind the prefix it is HBM (6.5 TB/s).  8 groups of 9 behind 16K tokens, 268 MB: 62 us, HBM
// (5.3 TB/s while attend runs; a slot's chain of S, softmax, P V is about 5000 cycles a block, and
// CTAs end 20% apart).  4 samples of a prompt of 1K tokens: 18 us, three launches of dependent loads
// and cold code.
#include <cfloat>
#include <cstring>

#include "kt_internal.cuh"

namespace kt {
namespace {

constexpr int ROWS = 128;                // rows of a tile: the M of the tensor-core steps
constexpr int SLOTS = 2;                 // tiles (each with its own scores and output) a CTA
constexpr int SOFT_WARPS = 8;            // a thread a row
constexpr int BOX = BS * 64 * 2;         // 128 tokens (or rows) x 64 channels, binary16
constexpr int TILE = 2 * BOX;            // 128 x 128
constexpr int PLAN_THREADS = 1024;

struct Item {      // blocks of one K/V head that a set of rows attends, for every K/V head
  int seq;         // whose table row to read
  int start;       // first block
  int blocks;
  int rows;        // B items: at most ROWS; A items (two tiles): at most 2 * ROWS
  int member;      // first row's place in the list of members times G, -1: seq's own rows
  int tokens;      // tokens of seq from block `start` on
  int row_base;    // B items: first row of the item's parts (head 0)
  int cum;         // steps of the items before
};

struct SeqPlan {   // where the parts of a sequence's rows are
  int item, r0, rows, pairs;  // B item of its own blocks; its first row among its group's rows
                              // (-1: nothing shared), those, and the group's first A item
  int single, pad[3];         // the group's B item
};

struct Head {      // A and B items: their steps, and the cost that is shared out
  int items_a, steps_a, cost_a;
  int items_b, steps_b, cost_b;
};

// Offsets in the workspace's part.
struct PrefixWs {
  size_t head, items_a, items_b, cost_a, cost_b, q_rows, seqs, parts, stats, total;
  long long rows_a;  // parts of A items come first
};

struct Params {
  CUtensorMap kmap, vmap;
  const __half* q;
  const float* k_scale;  // 8-bit cache
  const float* v_scale;
  const int32_t* table;
  const int32_t* seq_lens;
  const int32_t* cu;
  const int32_t* prefix;
  float* out;
  int* status;
  Head* head;
  Item* items_a;
  Item* items_b;
  int* cost_a;     // cost of the items before
  int* cost_b;
  int* q_rows;     // of members' rows: row of q (head 0)
  SeqPlan* seqs;   // [B]
  float* parts;    // of n rows: [32][n][4], the groups of four channels of all rows
  float2* stats;   // [rows]: m (up to a constant), l
  long long rows_a;
  int B, H_kv, G, groups, max_blocks, P, ctas, row_max;
  float scale_log2;
};

// What the kernel ahead has written is read past L1.
__device__ __forceinline__ Item load_item(const Item* p) {
  const int4 a = __ldcg(reinterpret_cast<const int4*>(p));
  const int4 b = __ldcg(reinterpret_cast<const int4*>(p) + 1);
  return Item{a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
}
__device__ __forceinline__ Head load_head(const Head* p) {
  const int* v = reinterpret_cast<const int*>(p);
  return Head{__ldcg(v), __ldcg(v + 1), __ldcg(v + 2), __ldcg(v + 3), __ldcg(v + 4), __ldcg(v + 5)};
}

__device__ __forceinline__ float ex2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// ---- plan --------------------------------------------------------------------------------
// The kernel runs its code once, and fetching it is what takes the time: few instructions, loops
// that are not unrolled.
struct PlanShared {
  int cu[MAX_SEGS + 1];
  int prefix[MAX_SEGS];
  int count[MAX_SEGS];          // members of group g
  int len[MAX_SEGS];
  int start[MAX_SEGS];          // prefix blocks that sequence b holds (0: no member)
  int group[MAX_SEGS];
  int4 seq_at[MAX_SEGS];        // exclusive sums over sequences: members, blocks, runs of their own
  int4 group_at[MAX_SEGS];      // over groups: A and B items (16 bits each), steps of both, rows of B
  int4 warp_sum[2][PLAN_THREADS / 32];
  int bad;
};

__device__ __forceinline__ int4 add4(int4 a, int4 b) {
  return make_int4(a.x + b.x, a.y + b.y, a.z + b.z, a.w + b.w);
}
// Inclusive sums over a warp.
__device__ __noinline__ int4 warp_scan4(int4 v) {
  const int lane = threadIdx.x & 31;
#pragma unroll 1
  for (int o = 1; o < 32; o <<= 1) {
    const int4 u = make_int4(__shfl_up_sync(0xffffffffu, v.x, o), __shfl_up_sync(0xffffffffu, v.y, o),
                             __shfl_up_sync(0xffffffffu, v.z, o), __shfl_up_sync(0xffffffffu, v.w, o));
    if (lane >= o) v = add4(v, u);
  }
  return v;
}

// A group's rows in tiles of 128, two at a time (A items), a last single one a B item.
struct Tiles {
  int rows, pairs, single;
  __device__ __forceinline__ Tiles(int members, int G)
      : rows(members >= 2 ? members * G : 0),
        pairs((rows + ROWS - 1) / ROWS / 2),
        single((rows + ROWS - 1) / ROWS & 1) {}
};

// Launched with as many threads as there are sequences or groups, at most PLAN_THREADS.
__global__ void __launch_bounds__(PLAN_THREADS) plan_kernel(const __grid_constant__ Params p) {
  extern __shared__ __align__(16) uint8_t plan_smem[];
  PlanShared& sh = *reinterpret_cast<PlanShared*>(plan_smem);
  const int tid = threadIdx.x, threads = blockDim.x, lane = tid & 31, warp = tid >> 5;
  if (tid == 0) sh.bad = 0;
  griddep_wait();
  griddep_launch_dependents();
  const int most = max(p.B, p.groups + 1);
#pragma unroll 1
  for (int i = tid; i < most; i += threads) {
    if (i <= p.groups) sh.cu[i] = p.cu[i];
    if (i < p.groups) {
      sh.prefix[i] = p.prefix[i];
      sh.count[i] = 0;
    }
    if (i < p.B) sh.len[i] = p.seq_lens[i];
  }
  __syncthreads();
  const int limit = p.max_blocks * BS;
#pragma unroll 1
  for (int i = tid; i < most; i += threads) {
    if (i <= p.groups) {
      const int c = sh.cu[i];
      if (c < 0 || c > p.B || (i > 0 && c < sh.cu[i - 1])) sh.bad = 1;  // nothing is shared then
    }
    if (i < p.groups && (sh.prefix[i] < 0 || sh.prefix[i] > p.max_blocks)) {
      set_status(p.status, KT_ERR_DEVICE_CHECK);
      sh.prefix[i] = 0;
    }
    if (i < p.B && (sh.len[i] < 0 || sh.len[i] > limit)) {
      set_status(p.status, KT_ERR_DEVICE_CHECK);
      sh.len[i] = sh.len[i] < 0 ? 0 : limit;
    }
  }
  __syncthreads();
  if (sh.bad && tid == 0) set_status(p.status, KT_ERR_DEVICE_CHECK);
  // members: sequences that hold all blocks of their group's prefix
#pragma unroll 1
  for (int b = tid; b < p.B; b += threads) {
    int lo = 0, hi = p.groups + 1;  // the last group that begins at or before b
    while (lo + 1 < hi) {
      const int mid = (lo + hi) / 2;
      if (sh.cu[mid] <= b) lo = mid;
      else hi = mid;
    }
    int start = 0;
    if (!sh.bad && lo < p.groups && sh.cu[lo] <= b) start = sh.prefix[lo];
    if (sh.len[b] < start * BS) start = 0;
    if (start > 0) atomicAdd(&sh.count[lo], 1);
    sh.start[b] = start;
    sh.group[b] = lo;
  }
  __syncthreads();
  // sums over sequences and over groups
  int4 seqs = make_int4(0, 0, 0, 0), groups = seqs;
#pragma unroll 1
  for (int i0 = 0; i0 < most; i0 += threads) {
    const int i = i0 + tid;
    int4 x[2] = {make_int4(0, 0, 0, 0), make_int4(0, 0, 0, 0)};
    if (i < p.B) {
      int start = sh.start[i];
      if (start > 0 && sh.count[sh.group[i]] < 2) sh.start[i] = start = 0;
      const int own = (sh.len[i] + BS - 1) / BS - start;
      x[0] = make_int4(start > 0, own, own > 0, 0);
    }
    if (i < p.groups) {
      const Tiles t(sh.count[i], p.G);
      const int blocks = sh.prefix[i];
      x[1] = make_int4(t.pairs << 16 | t.single, t.pairs * blocks, t.single * blocks,
                       t.single ? t.rows - t.pairs * 2 * ROWS : 0);
    }
    int4 incl[2];
#pragma unroll 1
    for (int k = 0; k < 2; ++k) {
      incl[k] = warp_scan4(x[k]);
      if (lane == 31) sh.warp_sum[k][warp] = incl[k];
    }
    __syncthreads();
    if (warp < 2) {
      const int4 v = lane < threads / 32 ? sh.warp_sum[warp][lane] : make_int4(0, 0, 0, 0);
      sh.warp_sum[warp][lane] = warp_scan4(v);
    }
    __syncthreads();
    if (warp > 0) {
      incl[0] = add4(incl[0], sh.warp_sum[0][warp - 1]);
      incl[1] = add4(incl[1], sh.warp_sum[1][warp - 1]);
    }
    const int4 s = add4(seqs, incl[0]), g = add4(groups, incl[1]);
    if (i < p.B) sh.seq_at[i] = make_int4(s.x - x[0].x, s.y - x[0].y, s.z - x[0].z, 0);
    if (i < p.groups)
      sh.group_at[i] = make_int4(g.x - x[1].x, g.y - x[1].y, g.z - x[1].z, g.w - x[1].w);
    seqs = add4(seqs, sh.warp_sum[0][threads / 32 - 1]);
    groups = add4(groups, sh.warp_sum[1][threads / 32 - 1]);
    __syncthreads();
  }
  const int pairs = groups.x >> 16, singles = groups.x & 0xffff;
  if (tid == 0)
    *p.head = Head{pairs,         groups.y * p.H_kv,           (groups.y + pairs) * p.H_kv,
                   singles + p.B, (groups.z + seqs.y) * p.H_kv,
                   (groups.z + singles + seqs.y + seqs.z) * p.H_kv};
  // items and rows; an item's cost is its blocks and one for its run
#pragma unroll 1
  for (int i = tid; i < most; i += threads) {
    Item it;
    if (i < p.B) {
      const int4 at = sh.seq_at[i];
      const int start = sh.start[i], n = sh.len[i], g = sh.group[i];
      const int cum = groups.z + at.y;
      it.seq = i;
      it.start = start;
      it.blocks = (n + BS - 1) / BS - start;
      it.rows = p.G;
      it.member = -1;
      it.tokens = n - start * BS;
      it.row_base = (groups.w + i * p.G) * p.H_kv;
      it.cum = cum * p.H_kv;
      p.items_b[singles + i] = it;
      p.cost_b[singles + i] = (cum + singles + at.z) * p.H_kv;
      SeqPlan sp;
      sp.item = singles + i;
      sp.r0 = -1;
      sp.rows = sp.pairs = sp.single = 0;
      if (start > 0) {
        const int c0 = sh.seq_at[sh.cu[g]].x;  // members before the group
        sp.r0 = (at.x - c0) * p.G;
        sp.rows = sh.count[g] * p.G;
        sp.pairs = sh.group_at[g].x >> 16;
        sp.single = sh.group_at[g].x & 0xffff;
#pragma unroll 1
        for (int j = 0; j < p.G; ++j) p.q_rows[at.x * p.G + j] = i * p.H_kv * p.G + j;
        // its first member, for its items (a sequence that is no member does not use its place)
        if (sp.r0 == 0) sh.group[sh.cu[g]] = i;
      }
      p.seqs[i] = sp;
    }
  }
  __syncthreads();
#pragma unroll 1
  for (int i = tid; i < p.groups; i += threads) {
    const Tiles t(sh.count[i], p.G);
    const int4 at = sh.group_at[i];
    Item it;
    if (t.rows > 0) it.seq = sh.group[sh.cu[i]];
    it.start = 0;
    it.blocks = sh.prefix[i];
    it.tokens = it.blocks * BS;
    it.row_base = at.w * p.H_kv;
#pragma unroll 1
    for (int j = 0; j < t.pairs + t.single; ++j) {
      const bool a = j < t.pairs;
      const int n = a ? (at.x >> 16) + j : at.x & 0xffff, cum = a ? at.y + j * it.blocks : at.z;
      it.rows = min(a ? 2 * ROWS : ROWS, t.rows - j * 2 * ROWS);
      it.member = sh.seq_at[sh.cu[i]].x * p.G + j * 2 * ROWS;
      it.cum = cum * p.H_kv;
      (a ? p.items_a : p.items_b)[n] = it;
      (a ? p.cost_a : p.cost_b)[n] = (cum + n) * p.H_kv;
    }
  }
}

// Equal shares of the cost of all steps, one a block and one a run (its queries, its part: a run
// of one block takes about twice the time of a block in the middle of a long one), among up to n
// workers: the first ones have one more than the others.  With more workers than cost each has a
// block or, for a run's own, nothing (4 samples of 1K tokens: 1.3 us less than with no more workers
// than blocks, some of which then had two).
struct Shares {
  int n, each, more;
  __device__ __forceinline__ Shares(int workers, int cost) : n(min(workers, cost)) {
    each = n > 0 ? cost / n : 1;
    more = cost - n * each;
  }
  __device__ __forceinline__ int first(int w) const { return w * each + min(w, more); }
  __device__ __forceinline__ int worker_of(int x) const {
    const int cut = more * (each + 1);
    return x < cut ? x / (each + 1) : more + (x - cut) / each;
  }
};

// The number of slot s among the workers of B steps: backwards, as the first CTAs may have one more
// A step than the others, and the first workers one more B step.
__device__ __forceinline__ int b_worker(const Params& p, int s) {
  return s * p.ctas + p.ctas - 1 - (int)blockIdx.x;
}

struct Start {     // where a CTA (A) or a slot (B; slot s: worker b_worker) begins
  Item first;      // its first item, that one's number, a head and a block of it
  int item, head, block;
  int step;        // its number among all steps
};

// The place of worker w's first step, found by a warp; its share is what lies before w + 1's.
__device__ __noinline__ Start find_start(const Item* items, const int* cost, int n_items,
                                         const Shares shares, int steps, int w) {
  const int lane = threadIdx.x & 31;
  Start s;
  s.item = s.head = s.block = 0;
  s.step = steps;
  if (w >= shares.n) return s;
  const int x = shares.first(w);
  int lo = 0, n = n_items, at = 0;  // the last item with cost <= x: never one without blocks
#pragma unroll 1
  while (n > 1) {
    const int stride = (n + 31) / 32, i = lane * stride;
    const int c = i < n ? __ldcg(cost + lo + i) : 0x7fffffff;
    const int k = __popc(__ballot_sync(0xffffffffu, c <= x)) - 1;
    lo += k * stride;
    n = min(stride, n - k * stride);
  }
  at = __ldcg(cost + lo);
  s.first = load_item(items + lo);
  s.item = lo;
  s.head = (x - at) / (s.first.blocks + 1);
  // the first unit of a run's cost is its own, then its blocks
  s.block = max(0, x - at - s.head * (s.first.blocks + 1) - 1);
  s.step = s.first.cum + s.head * s.first.blocks + s.block;
  return s;
}

// ---- attend ------------------------------------------------------------------------------
// Warps 0-7 hold the rows, a thread a row: warp w has slot w / 4 and the 32 TMEM lanes of
// quarter w % 4.  Warps 8 and 9 issue the tensor-core steps of a slot each, so that one slot's
// fill the pauses of the other's; warp 10 loads K and V tiles into a ring of 32 KB entries;
// warp 11 fetches the queries of the next run of blocks.  A run of up to 64 rows takes one
// half of the slot's 128 in turn with the next one, so that its queries come while the other
// half's are in use.  (Two threads a row have 104 registers each for half an output row and a
// chunk of scores, and spill: 4400 cycles a softmax instead of 1900.)
//
// A slot's block: S (TMEM, 128 columns) = Q K^T; the row threads turn it into P, which goes
// where the last block's output was; O = P V takes the place of S; the row threads add it to
// their running output in registers, out = out * alpha + O, and the next S takes the place of
// P.  So a block's P V is summed apart from the running output, no output is rescaled in
// TMEM, and the scores stay until P is whole: the exponentials use the running maximum of the
// blocks before (as h = 8 - maximum, one rounded number that all blocks' p share) and are made
// again, after a search for the block's own, where their sum shows that one may not fit binary16
// (alpha then scales what was summed before).  Where there is no maximum yet it is taken first.
//
// P is held as two binary16, 2^8 p = hi - lo (22 bits; steps of at least 2^-24), and
// P V as two products (the tensor cores negate lo): with one alone the output would be good to 11
// bits only, and it is binary32.  For 16 tokens, the K of a tensor-core step, columns 0-7 are hi,
// 8-15 lo.
//
// A items (two tiles of rows over the same blocks) go through both slots at once, each K/V
// tile read once; with B items the slots are on their own, each with its own share.
struct Unit {      // a run of blocks of one (item, head) in a slot
  int rows, row0;  // the slot's rows row0 .. row0 + rows - 1
  int run;         // blocks
  int tokens;      // tokens from its first block on
  long long part;  // its part's first row in the workspace
};
// A run's queries are fetched once the tensor cores are done with those of the run before
// last (their half): all row warps have then arrived for a block of the run before that, so
// they have read the description before, whose place in four the new one takes.
constexpr int UNITS = 4;
constexpr int STEPS_AHEAD = 8;  // steps described: more than the rings hold

// The 8-bit cache: its codes arrive in a ring of their own, and four more warps (12-15) turn each
// tile into a binary16 one in the ring that the tensor cores read.  Two tiles of codes are all that
// the shared memory has room for beside four of binary16, so one more waits in those warps'
// registers for the end of its entry's last use, and the tiles after them are fetched into L2 ahead
// of their loads (32 sequences behind 128K tokens: 164 us with the codes left in shared memory until
// then, 142 with one tile in registers, and 142 with three entries and four tiles of codes).
template <bool F8>
struct Config {
  static constexpr int entries = F8 ? 4 : 5;  // K or V tiles that the tensor cores read
  static constexpr int codes = F8 ? 2 : 0;    // tiles of codes
  static constexpr int threads = (SOFT_WARPS + (F8 ? 8 : 4)) * 32;
  // Registers pass from the other warps to the row threads.  The three (four) warpgroups are
  // launched with as many a thread as the compiler took (168 and 128), in eights; the shares must
  // not add up to more than those, or the row threads would wait for registers for ever, and each
  // must lie on its side of them.  The host checks it before the first launch.
  static constexpr int row_regs = F8 ? 192 : 216, control_regs = F8 ? 64 : 72;
  static constexpr bool registers_ok(int taken) {
    const int launched = (taken + 7) / 8 * 8, others = F8 ? 2 : 1;
    return control_regs <= launched && launched <= row_regs &&
           2 * row_regs + others * control_regs <= (2 + others) * launched;
  }
};
static_assert(Config<false>::registers_ok(168) && Config<false>::registers_ok(161) &&
                  Config<false>::registers_ok(216) && !Config<false>::registers_ok(160) &&
                  !Config<false>::registers_ok(217),
              "more registers than needed are no error, fewer are");
static_assert(Config<true>::registers_ok(128) && Config<true>::registers_ok(121) &&
                  Config<true>::registers_ok(192) && !Config<true>::registers_ok(120) &&
                  !Config<true>::registers_ok(193),
              "more registers than needed are no error, fewer are");
constexpr int CODE_TILE = BS * D;
constexpr int FETCH_AHEAD = 4;  // steps of a slot fetched into L2 ahead of their loads

struct Step {
  int bad;                // the page is outside the pool (or a scale is out of range)
  int valid;              // tokens
  float k_scale, v_scale;
  int slot;               // whose `full` barriers say that its tiles are there (A steps: 0) ...
  uint32_t v_parity;      // ... and the parity of V's
};
template <bool F8>
struct Misc {
  // An entry has a barrier `full` for each slot: a slot does not wait for the tiles of the other
  // one, and on a barrier that both share it would take the phase before the last for its own
  // when a tile of the other's is late (tiles do not arrive in order).
  uint64_t full[SLOTS][Config<F8>::entries], empty[Config<F8>::entries];
  uint64_t code_full[F8 ? Config<F8>::codes : 1], code_empty[F8 ? Config<F8>::codes : 1];
  uint64_t s_full[SLOTS], p_full[SLOTS], o_full[SLOTS];
  uint64_t q_full[SLOTS][UNITS], q_done[SLOTS][2];
  uint64_t a_done;               // the A steps have been issued
  Unit unit[SLOTS][UNITS];
  uint32_t tmem;
  Step step[STEPS_AHEAD];
  Start start[1 + SLOTS][2];     // of the A share and the slots' B shares, and of the next worker
};
template <bool F8>
constexpr int smem_bytes() {
  return SLOTS * TILE + Config<F8>::entries * TILE + Config<F8>::codes * CODE_TILE + sizeof(Misc<F8>);
}
static_assert(smem_bytes<false>() <= 232448 && smem_bytes<true>() <= 232448, "shared memory of a CTA");
static_assert(smem_bytes<false>() > 233472 / 2, "one CTA an SM: it holds all of TMEM");
constexpr uint32_t TMEM_COLS = 512;

// Columns of this thread's TMEM lane: loads without their wait (a register of an earlier load
// may be used behind tmem_wait_ld, which names it), and stores.
__device__ __forceinline__ void tmem_ld16_async(uint32_t taddr, float (&v)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,"
      "%14,%15}, [%16];"
      : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]),
        "=f"(v[7]), "=f"(v[8]), "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]),
        "=f"(v[14]), "=f"(v[15])
      : "r"(taddr));
}
__device__ __forceinline__ void tmem_wait_ld(float (&v)[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+f"(v[0]), "+f"(v[1]), "+f"(v[2]), "+f"(v[3]), "+f"(v[4]), "+f"(v[5]),
                 "+f"(v[6]), "+f"(v[7]), "+f"(v[8]), "+f"(v[9]), "+f"(v[10]), "+f"(v[11]),
                 "+f"(v[12]), "+f"(v[13]), "+f"(v[14]), "+f"(v[15])
               :
               : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,"
      "%13,%14,%15};" ::"r"(r[0]),
      "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
      "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_wait_st() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

// Two binary32 operations in one instruction.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{\n\t.reg .b64 x, y, z, w;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
      "mov.b64 z, {%6, %7};\n\tfma.rn.f32x2 w, x, y, z;\n\tmov.b64 {%0, %1}, w;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 x, y, w;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
      "add.rn.f32x2 w, x, y;\n\tmov.b64 {%0, %1}, w;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 x, y, w;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
      "mul.rn.f32x2 w, x, y;\n\tmov.b64 {%0, %1}, w;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// 2^8 p of 16 tokens as two binary16 each: rounded, and the rounding (hi - x, in one mixed-
// precision instruction on the FMA pipe; unpacking hi, or cutting x off, would go through the
// pipe that the conversions keep busy: 1880 cycles a block of two rows a lane instead of 1624).
__device__ __forceinline__ void split16(const float* x, uint32_t (&w)[16]) {
#pragma unroll
  for (int j = 0; j < 16; j += 2) {
    float a, b;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(w[j / 2]) : "f"(x[j + 1]), "f"(x[j]));
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\t"
        "sub.f32.f16 %0, l, %3;\n\tsub.f32.f16 %1, h, %4;\n\t}"
        : "=f"(a), "=f"(b)
        : "r"(w[j / 2]), "f"(x[j]), "f"(x[j + 1]));
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(w[8 + j / 2]) : "f"(b), "f"(a));
  }
}

// D[tmem] (+)= A[tmem] . B[sdesc]^T
__device__ __forceinline__ void umma_f16_ta(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc,
                                            bool accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(accumulate ? 1u : 0u)
      : "memory");
}

// A B operand whose rows in memory are K steps (V: a token's 64 channels in 128 swizzled
// bytes): 8 tokens are 1024 bytes, the other 64 channels lie a box further.
__device__ __forceinline__ uint64_t sdesc_mn_sw128(uint32_t saddr) {
  uint64_t d = (uint64_t)((saddr >> 4) & 0x3FFFu);
  d |= (uint64_t)(BOX >> 4) << 16;    // between the 64-channel boxes
  d |= (uint64_t)(1024u >> 4) << 32;  // between groups of 8 tokens
  d |= (uint64_t)1u << 46;
  d |= (uint64_t)2u << 61;
  return d;
}
constexpr uint32_t IDESC_S = umma_idesc_f16_f32(ROWS, BS);
constexpr uint32_t IDESC_O = umma_idesc_f16_f32(ROWS, D) | (1u << 16);  // B transposed
constexpr uint32_t NEGATE_A = 1u << 13;

// Scores of tokens from `valid` on leave the softmax; v holds those of tokens first ...
__device__ __forceinline__ void mask16(float (&v)[16], int first, int valid) {
#pragma unroll
  for (int j = 0; j < 16; ++j)
    if (first + j >= valid) v[j] = -INFINITY;
}

constexpr float SCALE_MIN = 0x1p-30f, SCALE_MAX = 0x1p30f;  // of the 8-bit cache

// log2 of the factor of P, and the largest sum of a block's 2^8 p whose terms surely are
// binary16 (65504 at most).
constexpr float P_SHIFT = 8.0f, SUM_MAX = 65000.0f;
// From here on (and where there is none yet) a row takes every block's own maximum, and the
// differences to it before they are scaled: next to 2^20 a binary32 shift is off by up to 2^-4,
// further up by so much that 2^8 p would leave binary16.
constexpr float BIG_SHIFT = 0x1p20f;

template <int N>
__device__ __forceinline__ void regs_inc() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void regs_dec() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

// The softmax runs over chunks of 16 columns, the next one's load in flight, two a turn of the
// loop: eight in a row are ten kilobytes of code, which every launch fetches anew (3300 cycles
// for its first block instead of 2500).
//
// A row's largest score (columns from taddr on).
template <bool MASK>
__device__ __forceinline__ float row_max(uint32_t taddr, int valid) {
  float v[2][16];
  float top = -INFINITY, top2 = -INFINITY;
  tmem_ld16_async(taddr, v[0]);
  tmem_wait_ld(v[0]);
#pragma unroll 1
  for (int c0 = 0; c0 < BS; c0 += 32) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int c = c0 + 16 * i;
      float(&x)[16] = v[i];
      tmem_ld16_async(taddr + min(c + 16, BS - 16), v[i ^ 1]);
      if (MASK) mask16(x, c, valid);
#pragma unroll
      for (int j = 0; j < 16; j += 4) {
        top = max3(top, x[j], x[j + 1]);
        top2 = max3(top2, x[j + 2], x[j + 3]);
      }
      tmem_wait_ld(v[i ^ 1]);
    }
  }
  return fmaxf(top, top2);
}

// 2^(s scale + shift) of a row's scores at `from`, in two parts to `to`; returns their sum.  BIG:
// 2^((s - s0) scale + shift).
// An element costs four issue slots (half an FMA and an addition of two, the exponential, two
// halves of conversions, a mixed-precision subtraction); the exponentials bound it, 4 cycles a
// warp's: 512 a block.
template <bool MASK, bool BIG>
__device__ __forceinline__ float row_exp(uint32_t from, uint32_t to, int valid, float2 scale2,
                                         float shift, float s0) {
  const float2 shift2 = make_float2(shift, shift);
  float2 sum[2] = {make_float2(0.0f, 0.0f), make_float2(0.0f, 0.0f)};
  float v[2][16];
  tmem_ld16_async(from, v[0]);
  tmem_wait_ld(v[0]);
#pragma unroll 1
  for (int c0 = 0; c0 < BS; c0 += 32) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int c = c0 + 16 * i;
      float(&x)[16] = v[i];
      tmem_ld16_async(from + min(c + 16, BS - 16), v[i ^ 1]);
      if (MASK) mask16(x, c, valid);
#pragma unroll
      for (int j = 0; j < 16; j += 2) {
        float2 y = make_float2(x[j], x[j + 1]);
        if (BIG) y = add2(y, make_float2(-s0, -s0));
        y = fma2(y, scale2, shift2);
        x[j] = ex2_fast(y.x);
        x[j + 1] = ex2_fast(y.y);
        sum[j / 2 & 1] = add2(sum[j / 2 & 1], make_float2(x[j], x[j + 1]));
      }
      uint32_t w16[16];
      split16(x, w16);
      tmem_wait_ld(v[i ^ 1]);
      tmem_st16(to + c, w16);
    }
  }
  return (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
}

// The same number in every lane, and known as such to the compiler.
__device__ __forceinline__ int uniform(int x) { return __reduce_max_sync(0xffffffffu, x); }
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}"
               : "=r"(r));
  return r != 0;
}
// mbar_wait by a whole warp, with the same answer in every lane.
__device__ __forceinline__ bool mbar_wait_warp(uint32_t bar, uint32_t parity, int* status,
                                               uint64_t limit = WAIT_LIMIT_NS) {
  if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
  const uint64_t t0 = globaltimer();
  for (uint32_t i = 1;; ++i) {
    if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
    if ((i & 255u) == 0 && __any_sync(0xffffffffu, globaltimer() - t0 > limit)) {
      set_status(status, KT_ERR_TIMEOUT);
      return false;
    }
  }
}

// A walk over the steps of a share: runs of blocks of one (item, head).
struct Walk {
  const Item* items;
  Item it;                      // the item at hand
  int item, head, block, left;  // `left` steps of the share
};
__device__ __forceinline__ Walk walk_of(const Item* items, const Start* s) {
  return Walk{items, s[0].first, s[0].item, s[0].head, s[0].block, s[1].step - s[0].step};
}
__device__ __forceinline__ int run_of(const Walk& w) { return min(w.left, w.it.blocks - w.block); }
// To the next run, behind one of `run` blocks.
__device__ __forceinline__ void advance(Walk& w, int run, int heads) {
  w.left -= run;
  w.block = 0;
  if (++w.head < heads || w.left == 0) return;
  w.head = 0;
  do {
    w.it = load_item(w.items + ++w.item);
  } while (w.it.blocks == 0);
}

// First ring entry of slot s's B step k (K; V is the next one), behind `a` A steps: the
// slots' steps take turns as long as both have some.
__device__ __forceinline__ int entry_b(int s, int k, int a, int other) {
  return 2 * (a + k + min(s == 0 ? k : k + 1, other));
}

// Parity of the n-th use of an entry of a ring of N.
template <int N>
__device__ __forceinline__ uint32_t ring_parity(int n) {
  return (uint32_t)(n / N) & 1u;
}

// L2 prefetch of a tile.
__device__ __forceinline__ void tma_prefetch_2d(const CUtensorMap* map, int x, int y) {
  asm volatile("cp.async.bulk.prefetch.tensor.2d.L2.global.tile [%0, {%1, %2}];" ::"l"(
                   reinterpret_cast<uint64_t>(map)),
               "r"(x), "r"(y)
               : "memory");
}

// A tile of codes (128-byte swizzled rows of 128 codes) into a tile of binary16 (two boxes of 64
// channels) by 128 threads, 16 codes at a time: a warp has one of the boxes, eight rows at a time,
// four lanes a row.  Eight lanes have rows r and r ^ 5, whose 16-byte words are in different banks
// both as codes (bit 2) and as binary16 (bit 0).
constexpr int CODE_WORDS = BS / 16;
struct CodeLane {
  int row, from, to;  // first row (the others are 16 apart), bytes into the tiles
  __device__ __forceinline__ explicit CodeLane(int t) {
    const int box = t >> 5 & 1, c = t & 3, r = (t >> 3 & 3) ^ (t >> 2 & 1) * 5;
    row = (t >> 6) * 8 + r;
    from = row * 128 + (((box * 4 + c) ^ r) << 4);
    to = box * BOX + row * 128 + (((2 * c) ^ r) << 4);
  }
};
__device__ __forceinline__ void load_codes(const uint8_t* code, CodeLane at, uint4 (&v)[CODE_WORDS]) {
#pragma unroll
  for (int i = 0; i < CODE_WORDS; ++i)
    v[i] = *reinterpret_cast<const uint4*>(code + at.from + i * (16 * 128));
}
// Rows from `valid` on become zeros.
__device__ __forceinline__ void store_codes(uint8_t* tile, int valid, CodeLane at,
                                            uint4 (&v)[CODE_WORDS]) {
  if (valid < BS) {
#pragma unroll
    for (int i = 0; i < CODE_WORDS; ++i)
      if (at.row + 16 * i >= valid) v[i] = make_uint4(0, 0, 0, 0);
  }
  uint8_t* to = tile + at.to;
  uint8_t* to2 = tile + (at.to ^ 16);
#pragma unroll
  for (int i = 0; i < CODE_WORDS; ++i) {
    *reinterpret_cast<uint4*>(to + i * (16 * 128)) =
        make_uint4(f8x2_lo(v[i].x), f8x2_hi(v[i].x), f8x2_lo(v[i].y), f8x2_hi(v[i].y));
    *reinterpret_cast<uint4*>(to2 + i * (16 * 128)) =
        make_uint4(f8x2_lo(v[i].z), f8x2_hi(v[i].z), f8x2_lo(v[i].w), f8x2_hi(v[i].w));
  }
}

// Queries of a run into two swizzled boxes (chunk c of row i: box c / 8, slot (c % 8) ^ (i % 8)).
// A lane finds where four of the rows are; then 16 lanes copy a row, two rows at a time.
__device__ __forceinline__ void load_queries(const Params& p, const Item& it, int head, int off,
                                             int rows, uint32_t q, int row0, int lane) {
  int at[ROWS / 32];  // rows of q
#pragma unroll
  for (int j = 0; j < ROWS / 32; ++j) {
    const int i = min(j * 32 + lane, rows - 1);
    at[j] = (it.member >= 0 ? __ldcg(p.q_rows + it.member + off + i) : it.seq * p.H_kv * p.G + i) +
            head * p.G;
  }
  const int c = lane & 15, odd = lane >> 4;
  const char* src = reinterpret_cast<const char*>(p.q) + c * 16;
  const uint32_t dst = q + (c >> 3) * BOX + (row0 + odd) * 128;  // row0 is a multiple of 8
#pragma unroll
  for (int j = 0; j < ROWS / 32; ++j) {
#pragma unroll 1
    for (int i0 = 0; i0 < 32 && j * 32 + i0 < rows; i0 += 8) {
#pragma unroll
      for (int i = 0; i < 8; i += 2) {  // behind the last row that one again
        const int row = __shfl_sync(0xffffffffu, at[j], i0 + i + odd);
        cp_async_16(dst + (j * 32 + i0 + i) * 128 + (((c & 7) ^ (i + odd)) << 4),
                    src + (size_t)row * (D * 2));
      }
    }
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
  fence_proxy_async_smem();
  __syncwarp();
}

template <bool F8>
__global__ void __launch_bounds__(Config<F8>::threads, 1)
    attend_kernel(const __grid_constant__ Params p) {
  constexpr int ENTRIES = Config<F8>::entries, CODES = F8 ? Config<F8>::codes : 1;
  extern __shared__ __align__(1024) uint8_t smem[];
  uint8_t* codes = smem + (SLOTS + ENTRIES) * TILE;
  Misc<F8>& ms = *reinterpret_cast<Misc<F8>*>(codes + Config<F8>::codes * CODE_TILE);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int cta = blockIdx.x;
  const uint32_t sQ = smem_u32(smem), ring = sQ + SLOTS * TILE;
  const uint32_t full = smem_u32(ms.full), empty = smem_u32(ms.empty);
  const uint32_t s_full = smem_u32(ms.s_full), p_full = smem_u32(ms.p_full);
  const uint32_t o_full = smem_u32(ms.o_full);
  const uint32_t q_full = smem_u32(ms.q_full), q_done = smem_u32(ms.q_done);
  const uint32_t code_full = smem_u32(ms.code_full), code_empty = smem_u32(ms.code_empty);
  if (tid == 0) {
    for (int i = 0; i < ENTRIES; ++i) {
      mbar_init(empty + 8 * i, 2);
    }
    // (arrivals of four converting warps, or of the load)
    for (int i = 0; i < SLOTS * ENTRIES; ++i) mbar_init(full + 8 * i, F8 ? 4 : 1);
    for (int i = 0; i < CODES; ++i) {
      mbar_init(code_full + 8 * i, 1);
      mbar_init(code_empty + 8 * i, 4);
    }
    for (int i = 0; i < SLOTS; ++i) {
      mbar_init(s_full + 8 * i, 1);
      mbar_init(p_full + 8 * i, SOFT_WARPS / SLOTS);
      mbar_init(o_full + 8 * i, 1);
    }
    for (int i = 0; i < UNITS * SLOTS; ++i) mbar_init(q_full + 8 * i, 1);
    for (int i = 0; i < 2 * SLOTS; ++i) mbar_init(q_done + 8 * i, 1);
    mbar_init(smem_u32(&ms.a_done), 1);
    fence_mbar_init();
    prefetch_tensormap(&p.kmap);
    prefetch_tensormap(&p.vmap);
  }
  if (warp == SOFT_WARPS) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_u32(&ms.tmem)),
                 "r"(TMEM_COLS));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = ms.tmem;
  griddep_wait();
  griddep_launch_dependents();
  if (warp < 2 * (1 + SLOTS)) {
    // this CTA's shares: their beginnings and their ends
    const Head h = load_head(p.head);
    const bool a = warp < 2;
    const int n = a ? p.ctas : p.ctas * SLOTS, steps = a ? h.steps_a : h.steps_b;
    const int w = (a ? cta : b_worker(p, (warp >> 1) - 1)) + (warp & 1);
    const Shares shares(n, a ? h.cost_a : h.cost_b);
    const Start st = find_start(a ? p.items_a : p.items_b, a ? p.cost_a : p.cost_b,
                                a ? h.items_a : h.items_b, shares, steps, w);
    if (lane == 0) ms.start[warp >> 1][warp & 1] = st;
  }
  __syncthreads();
  const int na = ms.start[0][1].step - ms.start[0][0].step;
  const int all_steps = na + ms.start[1][1].step - ms.start[1][0].step + ms.start[2][1].step -
                        ms.start[2][0].step;

  // the bound of a wait for the end of a whole run: a step takes a few microseconds
  const uint64_t run_limit = WAIT_LIMIT_NS + (uint64_t)all_steps * 20000;

  if (warp >= SOFT_WARPS) {
  regs_dec<Config<F8>::control_regs>();
  if (warp == SOFT_WARPS + 2) {
    // ============================ K and V tiles ============================
    const uint64_t pol = l2_evict_first_policy();
    const int row_end = p.P * p.H_kv * BS;  // reads zeros
    constexpr int RING = F8 ? CODES : ENTRIES;
    int e = 0;
    uint32_t used[SLOTS] = {0, 0}, last = 0;  // parities of the entries' uses; the last one's slot
    bool ok = true;
    // (the scales of the 8-bit cache come with the pages: any value of [2^-30, 2^30])
    auto load = [&](int slot, int page, int head, int valid, float ks, float vs) {
      bool bad = page < 0 || page >= p.P;
      if (F8) bad = bad || !(ks >= SCALE_MIN && ks <= SCALE_MAX && vs >= SCALE_MIN && vs <= SCALE_MAX);
      const int row = bad ? row_end : (page * p.H_kv + head) * BS;
      if (lane == 0) {
        if (bad) set_status(p.status, KT_ERR_DEVICE_CHECK);
        ms.step[(e >> 1) % STEPS_AHEAD] =
            Step{bad, bad ? 0 : min(BS, valid), bad ? 1.0f : ks, bad ? 0.0f : vs, slot,
                 (slot ? used[1] : used[0]) >> ((e + 1) % ENTRIES) & 1u};
      }
#pragma unroll 1
      for (int side = 0; side < 2 && ok; ++side, ++e) {
        const CUtensorMap* map = side == 0 ? &p.kmap : &p.vmap;
        const int st = e % RING;
        const uint32_t landed = (F8 ? code_full : full + 8 * ENTRIES * slot) + 8 * st;
        if (e >= RING)
          ok = mbar_wait_warp((F8 ? code_empty : empty) + 8 * st, ring_parity<RING>(e) ^ 1, p.status);
        if (!ok) break;
        const uint32_t bit = 1u << (e % ENTRIES);
        if (slot) used[1] ^= bit, last |= bit;
        else used[0] ^= bit, last &= ~bit;
        if (lane == 0) {
          if (F8) {
            mbar_arrive_expect_tx(landed, CODE_TILE);
            tma_load_2d(smem_u32(codes) + st * CODE_TILE, map, 0, row, landed, pol);
          } else {
            const uint32_t dst = ring + st * TILE;
            mbar_arrive_expect_tx(landed, TILE);
            tma_load_2d(dst, map, 0, row, landed, pol);
            tma_load_2d(dst + BOX, map, 64, row, landed, pol);
          }
        }
        __syncwarp();
      }
    };
    struct Turn {
      Walk w;
      int slot, at, run, page;     // the pages of the run's next 32 blocks, one a lane
      float ks, vs;
    };
    auto turn = [&](Turn& t) {
      if (t.w.left == 0) return;
      if ((t.at & 31) == 0) {
        t.run = run_of(t.w);
        const int j = t.w.block + t.at + lane;
        t.page = -1;
        t.ks = t.vs = 0.0f;
        if (j < t.w.it.blocks)
          t.page = p.table[(size_t)t.w.it.seq * p.max_blocks + t.w.it.start + j];
        if (F8 && t.page >= 0 && t.page < p.P) {
          t.ks = p.k_scale[(size_t)t.page * p.H_kv + t.w.head];
          t.vs = p.v_scale[(size_t)t.page * p.H_kv + t.w.head];
        }
        if (F8 && lane < FETCH_AHEAD && t.at + lane < t.run && t.page >= 0 && t.page < p.P) {
          tma_prefetch_2d(&p.kmap, 0, (t.page * p.H_kv + t.w.head) * BS);
          tma_prefetch_2d(&p.vmap, 0, (t.page * p.H_kv + t.w.head) * BS);
        }
        __syncwarp();
      }
      const int i = t.at & 31;
      if (F8 && i + FETCH_AHEAD < 32 && t.at + FETCH_AHEAD < t.run && lane == i + FETCH_AHEAD &&
          t.page >= 0 && t.page < p.P) {
        tma_prefetch_2d(&p.kmap, 0, (t.page * p.H_kv + t.w.head) * BS);
        tma_prefetch_2d(&p.vmap, 0, (t.page * p.H_kv + t.w.head) * BS);
      }
      __syncwarp();
      load(t.slot, __shfl_sync(0xffffffffu, t.page, i), t.w.head,
           t.w.it.tokens - (t.w.block + t.at) * BS, F8 ? __shfl_sync(0xffffffffu, t.ks, i) : 1.0f,
           F8 ? __shfl_sync(0xffffffffu, t.vs, i) : 1.0f);
      if (++t.at == t.run) {
        advance(t.w, t.run, p.H_kv);
        t.at = 0;
      }
    };
    // A steps, then the slots' B steps in turn
    Turn t0 = {walk_of(p.items_a, ms.start[0]), 0, 0, 0, 0, 0.0f, 0.0f}, t1 = t0;
    t1.w.left = 0;
#pragma unroll 1
    for (int part = 0; part < 2; ++part) {
#pragma unroll 1
      while (ok && (t0.w.left > 0 || t1.w.left > 0)) {
        turn(t0);
        const Turn t = t0;
        t0 = t1;
        t1 = t;
        if (part == 0 || t0.w.left == 0) {  // (one walk only)
          t1 = t0;
          t0 = t;
        }
      }
      if (part == 0) {
        t0 = Turn{walk_of(p.items_b, ms.start[1]), 0, 0, 0, 0, 0.0f, 0.0f};
        t1 = Turn{walk_of(p.items_b, ms.start[2]), 1, 0, 0, 0, 0.0f, 0.0f};
        if (t0.w.left == 0) {
          const Turn t = t0;
          t0 = t1;
          t1 = t;
        }
      }
    }
    // nothing that arrives in this CTA's shared memory is in flight when it ends: loads, and the
    // tensor cores' arrivals when they are done with a tile (or queries), which come behind those
    // that let the rows finish
#pragma unroll 1
    for (int i = max(0, e - RING); i < e; ++i) {
      const int st = i % RING, slot = last >> st & 1;
      if (F8) {
        mbar_wait_warp(code_full + 8 * st, ring_parity<RING>(i), p.status);
      } else {
        const uint32_t parity = ((slot ? used[1] : used[0]) >> st & 1u) ^ 1u;
        mbar_wait_warp(full + 8 * (ENTRIES * slot + st), parity, p.status);
        mbar_wait_warp(empty + 8 * st, ring_parity<RING>(i), p.status);
      }
    }
  } else if (F8 && warp >= SOFT_WARPS + 4) {
    // ============================ codes to binary16 ============================
    const CodeLane at(tid - (SOFT_WARPS + 4) * 32);
    bool ok = true;
#pragma unroll 1
    for (int e = 0; e < 2 * all_steps && ok; ++e) {
      const int c = e % CODES, st = e % ENTRIES;
      ok = mbar_wait_warp(code_full + 8 * c, ring_parity<CODES>(e), p.status);
      if (!ok) break;
      const Step& step = ms.step[(e >> 1) % STEPS_AHEAD];
      const int valid = step.valid, slot = step.slot;
      uint4 v[CODE_WORDS];  // (the next load need not wait for the entry's last use)
      load_codes(codes + c * CODE_TILE, at, v);
      __syncwarp();
      if (lane == 0) mbar_arrive(code_empty + 8 * c);
      if (e >= ENTRIES) ok = mbar_wait_warp(empty + 8 * st, ring_parity<ENTRIES>(e) ^ 1, p.status);
      if (!ok) break;
      store_codes(smem + (SLOTS + st) * TILE, valid, at, v);
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(full + 8 * (ENTRIES * slot + st));
    }
#pragma unroll 1
    for (int e = max(0, 2 * all_steps - ENTRIES); e < 2 * all_steps; ++e)
          mbar_wait_warp(empty + 8 * (e % ENTRIES), ring_parity<ENTRIES>(e), p.status);
  } else if (warp == SOFT_WARPS + 3) {
    // ============================ runs and their queries ============================
    Walk w[SLOTS];
    int units[SLOTS] = {0, 0}, rows_before[SLOTS] = {0, 0};
    bool ok = true;
    for (int part = 0; part < 2 && ok; ++part) {
      const bool a = part == 0;
      w[0] = a ? walk_of(p.items_a, ms.start[0]) : walk_of(p.items_b, ms.start[1]);
      w[1] = a ? w[0] : walk_of(p.items_b, ms.start[2]);
      // a slot whose next run has no room yet does not hold up the other's: in the ring their
      // steps wait for one another
      uint64_t t0 = globaltimer();
      while (ok && (w[0].left > 0 || w[1].left > 0)) {
        bool moved = false;
#pragma unroll
        for (int s = 0; s < SLOTS; ++s) {
          if (w[s].left == 0) continue;
          const Item& it = w[s].it;
          const int off = a ? s * ROWS : 0, n = units[s], u = n % UNITS, buf = n & 1;
          const int rows = min(ROWS, it.rows - off);
          // the run before last is done with this half; a run of both halves waits for, and is
          // waited for by, its neighbours
          bool room = n < 2 || mbar_try_wait(q_done + 8 * (2 * s + buf), ((n >> 1) - 1) & 1);
          if (n >= 1 && (rows > ROWS / 2 || rows_before[s] > ROWS / 2))
            room = room && mbar_try_wait(q_done + 8 * (2 * s + (buf ^ 1)), ((n - 1) >> 1) & 1);
          if (!__all_sync(0xffffffffu, room)) continue;
          moved = true;
          const int run = run_of(w[s]);
          // the slots' halves differ, so that both keep other schedulers busy
          const int row0 = rows <= ROWS / 2 ? ((n + s) & 1) * (ROWS / 2) : 0;
          if (lane == 0) {
            Unit& unit = ms.unit[s][u];
            unit.rows = rows;
            unit.row0 = row0;
            unit.run = run;
            unit.tokens = it.tokens - w[s].block * BS;
            unit.part = a ? (cta + (long long)w[s].item * p.H_kv + w[s].head) * (2 * ROWS) + off
                          : p.rows_a + (long long)b_worker(p, s) * p.row_max + it.row_base +
                                (long long)w[s].head * it.rows;
          }
          load_queries(p, it, w[s].head, off, rows, sQ + s * TILE, row0, lane);
          if (lane == 0) mbar_arrive(q_full + 8 * (UNITS * s + u));
          __syncwarp();
          ++units[s];
          rows_before[s] = rows;
          advance(w[s], run, p.H_kv);
        }
        const uint64_t t = globaltimer();
        if (moved) t0 = t;
        else if (__any_sync(0xffffffffu, t - t0 > run_limit)) {
          if (lane == 0) set_status(p.status, KT_ERR_TIMEOUT);
          ok = false;
        }
      }
    }
#pragma unroll
    for (int s = 0; s < SLOTS; ++s)
#pragma unroll 1
      for (int n = max(0, units[s] - 2); n < units[s]; ++n)
        mbar_wait_warp(q_done + 8 * (2 * s + (n & 1)), (n >> 1) & 1, p.status);
  } else {
    // ============================ tensor-core steps ============================
    // The whole warp runs this, and what it loads goes through a warp reduction: the compiler
    // then keeps it in uniform registers, where the tensor-core instructions want their operands
    // (moving them there one by one took longer than the steps themselves).
    const bool leader = elect_one();
    const int na_u = uniform(na);
    const int nb0 = uniform(ms.start[1][1].step - ms.start[1][0].step);
    const int nb1 = uniform(ms.start[2][1].step - ms.start[2][0].step);
    bool ok = true;
    // K and V of A steps are waited for on slot 0's barriers, by both slots' steps
    const uint32_t tiles = full + 8 * ENTRIES * (warp - SOFT_WARPS);
    uint32_t used = 0;  // parities of the entries' uses
    // S = Q K^T of slot s's step k, once K, the run's Q and the end of the last P V are there;
    // n counts the runs begun, left the steps of the one at hand
    auto scores = [&](int s, int k, int e, bool both, int& n, int& left) {
      const int ek = e % ENTRIES;
      if (left == 0) {
        ok = ok && mbar_wait_warp(q_full + 8 * (UNITS * s + n % UNITS), (n / UNITS) & 1, p.status);
        left = uniform(ms.unit[s][n % UNITS].run);
        ++n;
      }
      ok = ok && mbar_wait_warp(tiles + 8 * ek, used >> ek & 1u, p.status) &&
           (k == 0 || mbar_wait_warp(o_full + 8 * s, (k - 1) & 1, p.status));
      if (!ok) return;
      if (!both || s == 1) used ^= 1u << ek;
      tc_fence_after();
      const uint64_t q = umma_sdesc_sw128(sQ + s * TILE), kb = umma_sdesc_sw128(ring + ek * TILE);
      const uint32_t st = tmem + s * 256 + (k & 1) * 128;
      --left;
      if (leader) {
#pragma unroll
        for (int ks = 0; ks < 8; ++ks) {
          const int at = ((ks >> 2) * BOX + (ks & 3) * 32) >> 4;
          umma_f16(st, q + at, kb + at, IDESC_S, ks > 0);
        }
        umma_commit(s_full + 8 * s);
        if (left == 0) umma_commit(q_done + 8 * (2 * s + (~n & 1)));  // the run's last use of Q
        umma_commit(empty + 8 * ek);
        if (!both) umma_commit(empty + 8 * ek);  // the other slot has no part in this one
      }
      __syncwarp();
    };
    // O = P V, the high and the low parts of P
    auto values = [&](int s, int k, int e, bool both) {
      const int ev = e % ENTRIES;
      ok = ok && mbar_wait_warp(tiles + 8 * ev, used >> ev & 1u, p.status) &&
           mbar_wait_warp(p_full + 8 * s, k & 1, p.status);
      if (!ok) return;
      if (!both || s == 1) used ^= 1u << ev;
      tc_fence_after();
      const uint64_t vb = sdesc_mn_sw128(ring + ev * TILE);
      const uint32_t st = tmem + s * 256 + (k & 1) * 128, pt = tmem + s * 256 + (~k & 1) * 128;
      if (leader) {
#pragma unroll
        for (int ks = 0; ks < 16; ++ks)
          umma_f16_ta(st, pt + (ks & 7) * 16 + (ks >> 3) * 8, vb + (ks & 7) * (2048 >> 4),
                      IDESC_O | (ks >= 8 ? NEGATE_A : 0u), ks > 0);
        umma_commit(o_full + 8 * s);
        umma_commit(empty + 8 * ev);
        if (!both) umma_commit(empty + 8 * ev);
      }
      __syncwarp();
    };
    // A steps: both slots from one warp, P V and the next scores of one in a row, so that the
    // softmax of each falls into the tensor-core time of the other.  (Two warps that issue as
    // operands come keep the slots in step, and the tensor cores idle meanwhile.)  Then B steps:
    // each slot from a warp of its own, at its own pace.
    int s = warp - SOFT_WARPS, n = 0, left = 0, n_other = 0, left_other = 0;
    if (s == 1) {  // the runs that the other warp issues
      Walk w = walk_of(p.items_a, ms.start[0]);
      for (; w.left > 0; ++n) advance(w, run_of(w), p.H_kv);
      n = uniform(n);
      // the barriers of those runs are past the phases before the first one waited for here
      if (na_u > 0) ok = mbar_wait_warp(smem_u32(&ms.a_done), 0, p.status, run_limit);
    }
    const int nb = s == 0 ? nb0 : nb1, other = s == 0 ? nb1 : nb0;
    int k = s == 0 ? 0 : na_u;
    if (k < na_u) {  // the first scores of both slots
#pragma unroll 1
      for (int x = 0; x < 2; ++x) {
        scores(x, 0, 0, true, n, left);
        const int t = n, u = left;
        n = n_other, left = left_other, n_other = t, left_other = u;
      }
    }
#pragma unroll 1
    while (ok && k < na_u + nb) {
      const bool a = k < na_u;
      // an A step: P V of step k and the scores of k + 1, slot by slot; a B step: its scores, P V
      const int e = a ? 2 * k : entry_b(s, k - na_u, na_u, other);
      if (!a) scores(s, k, e, false, n, left);
      values(s, k, e + 1, a);
      if (a && k + 1 < na_u) scores(s, k + 1, e + 2, true, n, left);
      if (a) {
        const int t = n, u = left;
        n = n_other, left = left_other, n_other = t, left_other = u;
        s ^= 1;
        if (s == 0 && ++k == na_u && lane == 0) mbar_arrive(smem_u32(&ms.a_done));
      } else {
        ++k;
      }
    }
    __syncwarp();
  }
  } else {
    // ============================ rows ============================
    regs_inc<Config<F8>::row_regs>();
    const int s = warp >> 2, quarter = warp & 3;
    const int r = quarter * 32 + lane;       // this thread's row of the slot
    const uint32_t tb = tmem + s * 256 + ((uint32_t)(quarter * 32) << 16);
    const int steps = na + ms.start[1 + s][1].step - ms.start[1 + s][0].step;
    const int other = ms.start[2 - s][1].step - ms.start[2 - s][0].step;
    bool ok = true;
    for (int k = 0, n = 0; k < steps && ok; ++n) {
      ok = mbar_wait_warp(q_full + 8 * (UNITS * s + n % UNITS), (n / UNITS) & 1, p.status);
      if (!ok) break;
      const Unit unit = ms.unit[s][n % UNITS];
      const int q0 = unit.row0 / 32, warps = (unit.row0 + unit.rows + 31) / 32 - q0;
      const int end = k + unit.run;
      if (quarter < q0 || quarter >= q0 + warps) {
        // no rows here; the warp keeps in step by arriving for each block (behind its loads from
        // tensor memory of the run before, whose columns the next products write)
        tc_fence_before();
        for (; k < end && ok; ++k) {
          ok = mbar_wait_warp(s_full + 8 * s, k & 1, p.status);
          if (ok && lane == 0) mbar_arrive(p_full + 8 * s);
        }
        continue;
      }
      const bool mine = r >= unit.row0 && r < unit.row0 + unit.rows;
      int tokens = unit.tokens;
      float acc[D], h = INFINITY, l = 0.0f;  // p = 2^(score + h - P_SHIFT)
#pragma unroll
      for (int i = 0; i < D; ++i) acc[i] = 0.0f;
      for (; k < end; ++k, tokens -= BS) {
        int valid = min(BS, tokens);
        const int e = k < na ? 2 * k : entry_b(s, k - na, na, other);
        const volatile Step* step = &ms.step[(e >> 1) % STEPS_AHEAD];
        const uint32_t ts = tb + (k & 1) * 128, tp = tb + (~k & 1) * 128;
        ok = mbar_wait_warp(s_full + 8 * s, k & 1, p.status);
        if (!ok) break;
        tc_fence_after();
        if (!F8 && valid < BS) {
          // V behind the last token may be anything, and 0 * NaN is NaN: zeros there
          const int ev = (e + 1) % ENTRIES;
          ok = mbar_wait_warp(full + 8 * ((k < na ? 0 : ENTRIES * s) + ev), step->v_parity, p.status);
          if (!ok) break;
          uint8_t* v = smem + SLOTS * TILE + ev * TILE;
          for (int idx = valid * 8 + (quarter - q0) * 32 + lane; idx < BS * 8; idx += warps * 32) {
            *reinterpret_cast<uint4*>(v + idx * 16) = make_uint4(0, 0, 0, 0);
            *reinterpret_cast<uint4*>(v + BOX + idx * 16) = make_uint4(0, 0, 0, 0);
          }
          fence_proxy_async_smem();
        }
        if (step->bad) valid = 0;
        float scale = p.scale_log2, v_scale = 1.0f;
        if (F8) {
          scale = fmaxf(scale * step->k_scale, FLT_MIN);  // (0 times a masked score is no number)
          v_scale = step->v_scale;
        }
        const float2 scale2 = make_float2(scale, scale);
        float sum = 0.0f, alpha = 1.0f, s0 = 0.0f, shift = h;
        // (a row takes a new maximum for its own need only: its numbers do not depend on others')
        bool need = mine && fabsf(h) >= BIG_SHIFT;
        for (int round = 0;; ++round) {
          bool big = false;
          if (__any_sync(0xffffffffu, need)) {
            const float top = valid < BS ? row_max<true>(ts, valid) : row_max<false>(ts, valid);
            if (need) {
              const float u = P_SHIFT - top * scale;
              if (u < h) {
                alpha = ex2_fast(u - h);  // 0 where there was nothing yet
                h = u;
              }
              shift = h;
              if (fabsf(u) >= BIG_SHIFT && fabsf(u) < INFINITY) {
                s0 = top;
                shift = P_SHIFT + (h - u);
              }
            }
            big = __any_sync(0xffffffffu, s0 != 0.0f);
          } else if (round > 0) {
            break;
          }
          if (h == INFINITY) shift = 0.0f;  // no token yet: all are masked
          if (round > 0) tmem_wait_st();  // the stores of P are not ordered among themselves
          if (big) {
            sum = valid < BS ? row_exp<true, true>(ts, tp, valid, scale2, shift, s0)
                             : row_exp<false, true>(ts, tp, valid, scale2, shift, s0);
          } else {
            sum = valid < BS ? row_exp<true, false>(ts, tp, valid, scale2, shift, s0)
                             : row_exp<false, false>(ts, tp, valid, scale2, shift, s0);
          }
          if (round > 0) break;
          need = mine && !need && sum > SUM_MAX;  // with its own maximum at most 128 * 2^8 = 2^15
        }
        l = fmaf(l, alpha, sum);
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(p_full + 8 * s);
        ok = mbar_wait_warp(o_full + 8 * s, k & 1, p.status);
        if (!ok) break;
        tc_fence_after();
        {
          if (__any_sync(0xffffffffu, alpha != 1.0f)) {  // (few blocks have a new maximum)
            const float2 alpha2 = make_float2(alpha, alpha);
#pragma unroll
            for (int i = 0; i < D; i += 2) {
              const float2 y = mul2(make_float2(acc[i], acc[i + 1]), alpha2);
              acc[i] = y.x;
              acc[i + 1] = y.y;
            }
          }
          const float2 v_scale2 = make_float2(v_scale, v_scale);
          float v[2][16];
          tmem_ld16_async(ts, v[0]);
          tmem_wait_ld(v[0]);
#pragma unroll
          for (int c = 0; c < D; c += 16) {
            float(&x)[16] = v[(c / 16) & 1];
            float(&next)[16] = v[(c / 16 + 1) & 1];
            if (c + 16 < D) tmem_ld16_async(ts + c + 16, next);
#pragma unroll
            for (int j = 0; j < 16; j += 2) {
              const float2 o = make_float2(x[j], x[j + 1]);
              const float2 y0 = make_float2(acc[c + j], acc[c + j + 1]);
              // (the V scale of the block is the O tile's)
              const float2 y = F8 ? fma2(o, v_scale2, y0) : add2(o, y0);
              acc[c + j] = y.x;
              acc[c + j + 1] = y.y;
            }
            if (c + 16 < D) tmem_wait_ld(next);
          }
        }
      }
      // this run's part of the rows: [32 groups of 4 channels][rows][4]
      const int rows = unit.rows, i = r - unit.row0;
      if (mine && ok) {
        const long long part = unit.part;
        float4* o = reinterpret_cast<float4*>(p.parts + part * D) + i;
#pragma unroll
        for (int c = 0; c < D / 4; ++c)
          o[(size_t)c * rows] = make_float4(acc[4 * c], acc[4 * c + 1], acc[4 * c + 2], acc[4 * c + 3]);
        p.stats[part + i] = make_float2(-h, l);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == SOFT_WARPS) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(TMEM_COLS));
  }
}

// ---- combine -----------------------------------------------------------------------------
// A warp takes 8 rows (consecutive ones of the batch, which mostly are of a tile too) and 16
// channels: its 8 x 16 bytes of a part's channel group are contiguous.  A row of a long prefix has
// a part for each CTA that met it (some 20 at 32K tokens): 16 of them in flight at a time (with 8,
// and the rest one by one, 32 sequences behind 128K tokens took 14 us here instead of 6).  It is
// bound by three round trips to L2: the sequence's place in the plan, its items, the parts (5 us
// with one of them, the plan read while attend still runs, which nothing promises to be there).
constexpr int COMBINE_WARPS = 8;
constexpr int COMBINE_ROWS = 8;
constexpr int COMBINE_BATCH = 16;  // parts in flight

__global__ void __launch_bounds__(COMBINE_WARPS * 32, 2)
    combine_kernel(const __grid_constant__ Params p) {
  const int lane = threadIdx.x & 31, all_rows = p.B * p.G;
  const int chunks = (all_rows + COMBINE_ROWS - 1) / COMBINE_ROWS;
  const int job = blockIdx.x * COMBINE_WARPS + (threadIdx.x >> 5);
  const int h = job / (chunks * 8), col = job % 8 * 4 + (lane >> 3);  // channels 4 col .. + 3
  const int row = job / 8 % chunks * COMBINE_ROWS + (lane & 7);
  if (h >= p.H_kv || row >= all_rows) return;
  const int b = row / p.G, g = row % p.G;
  griddep_wait();  // (also what the plan has written can be read from here on only)
  griddep_launch_dependents();
  const Head head = load_head(p.head);
  const int4 sp4 = __ldcg(reinterpret_cast<const int4*>(p.seqs + b));
  const SeqPlan sp = {sp4.x, sp4.y, sp4.z, sp4.w, __ldcg(&p.seqs[b].single), {0, 0, 0}};
  float M = -INFINITY, L = 0.0f;
  float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  // the prefix, then the sequence's own blocks: the parts of each worker that has steps of it
  int r = sp.r0 + g, off = 0, item = sp.item;
  bool a = false;
  if (sp.r0 >= 0) {
    const int pair = r / (2 * ROWS);
    a = pair < (sp.rows + ROWS - 1) / ROWS / 2;
    item = a ? sp.pairs + pair : sp.single;
    r -= pair * 2 * ROWS;
    off = r / ROWS * ROWS;
    r -= off;
  }
  Item it = load_item((a ? p.items_a : p.items_b) + item), own = load_item(p.items_b + sp.item);
  int cost = __ldcg((a ? p.cost_a : p.cost_b) + item);
  const int own_cost = __ldcg(p.cost_b + sp.item);
  const Shares shares_a(p.ctas, head.cost_a);
  const Shares shares_b(p.ctas * SLOTS, head.cost_b);
#pragma unroll 1
  for (int turn = sp.r0 >= 0 ? 0 : 1; turn < 2; ++turn) {
    if (turn == 1) {
      it = own;
      cost = own_cost;
      item = sp.item;
      r = g;
      off = 0;
      a = false;
    }
    if (it.blocks == 0) continue;
    const int rows = min(ROWS, it.rows - off);
    const int stride = a ? 2 * ROWS : p.row_max;
    const long long base = a ? (long long)(item * p.H_kv + h) * (2 * ROWS) + off
                             : p.rows_a + it.row_base + (long long)h * rows;
    const Shares& shares = a ? shares_a : shares_b;
    // the run's first unit of cost is its own, then its blocks
    const int x = cost + h * (it.blocks + 1) + 1;
    const int w0 = shares.worker_of(x), w1 = shares.worker_of(x + it.blocks - 1);
    for (int w = w0; w <= w1; w += COMBINE_BATCH) {
      float2 st[COMBINE_BATCH];
      float4 o[COMBINE_BATCH];
      float m = M;
#pragma unroll
      for (int i = 0; i < COMBINE_BATCH; ++i) {
        st[i] = make_float2(-INFINITY, 0.0f);
        o[i] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (w + i <= w1) {
          const long long first = base + (long long)(w + i) * stride;
          st[i] = __ldcg(p.stats + first + r);
          o[i] = __ldcg(reinterpret_cast<const float4*>(p.parts + first * D) + (size_t)col * rows + r);
        }
      }
#pragma unroll
      for (int i = 0; i < COMBINE_BATCH; ++i) m = fmaxf(m, st[i].x);
      const float ref = m == -INFINITY ? 0.0f : m, a0 = ex2_fast(M - ref);
      M = m;
      L *= a0;
      acc = make_float4(acc.x * a0, acc.y * a0, acc.z * a0, acc.w * a0);
#pragma unroll
      for (int i = 0; i < COMBINE_BATCH; ++i) {
        const float c = ex2_fast(st[i].x - ref);
        L = fmaf(st[i].y, c, L);
        acc.x = fmaf(o[i].x, c, acc.x);
        acc.y = fmaf(o[i].y, c, acc.y);
        acc.z = fmaf(o[i].z, c, acc.z);
        acc.w = fmaf(o[i].w, c, acc.w);
      }
    }
  }
  const float inv = L == 0.0f ? 0.0f : 1.0f / L;
  float* out = p.out + ((size_t)b * p.H_kv * p.G + h * p.G + g) * D;
  reinterpret_cast<float4*>(out)[col] =
      make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv);
}

// Its CTAs start as those of attend end; without a limit the first SMs that are free take them
// all, eight each.  The shared memory that they ask for (and do not use) leaves room for an even
// share an SM.
size_t combine_smem(int grid, int sms) {
  constexpr int SM_BYTES = 233472, CTA_BYTES = 1024;  // of an SM; what a CTA takes beside its own
  const int share = (grid + sms - 1) / sms;
  return share >= 8 ? 0 : (size_t)(SM_BYTES / share / 1024 * 1024 - CTA_BYTES);
}

PrefixWs prefix_layout(int B, int H_kv, int G) {
  PrefixWs L;
  const size_t rows = (size_t)B * H_kv * G;
  const int row_max = B * G < ROWS ? B * G : ROWS;
  const size_t max_pairs = (size_t)B * G / (ROWS + 1) + 1;
  size_t off = 0;
  L.head = off;
  off = align256(off + sizeof(Head));
  L.items_a = off;
  off = align256(off + max_pairs * sizeof(Item));
  L.items_b = off;
  off = align256(off + 2 * (size_t)B * sizeof(Item));
  L.cost_a = off;
  off = align256(off + max_pairs * 4);
  L.cost_b = off;
  off = align256(off + 2 * (size_t)B * 4);
  L.q_rows = off;
  off = align256(off + (size_t)B * G * 4);
  L.seqs = off;
  off = align256(off + (size_t)B * sizeof(SeqPlan));
  // A items: 256 rows for each (CTA, item and head) that meet; there are fewer than CTAs +
  // items of those.  B items: row_max rows a slot and the rows of all items.
  L.rows_a = B * G > ROWS ? (long long)(PREFIX_MAX_CTAS + max_pairs * H_kv) * 2 * ROWS : 0;
  const size_t total_rows = L.rows_a + (size_t)PREFIX_MAX_CTAS * SLOTS * row_max + 2 * rows;
  L.parts = off;
  off = align256(off + total_rows * D * 4);
  L.stats = off;
  off = align256(off + total_rows * 8);
  L.total = off;
  return L;
}

template <class P>
cudaError_t launch(void (*kernel)(P), const P& p, int grid, int threads, size_t smem,
                   cudaStream_t stream) {
  cudaLaunchConfig_t cfg;
  std::memset(&cfg, 0, sizeof(cfg));
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

template <bool F8>
cudaError_t prepare_attend() {
  cudaFuncAttributes attr;
  const cudaError_t r = cudaFuncGetAttributes(&attr, attend_kernel<F8>);
  if (r != cudaSuccess) return r;
  if (!Config<F8>::registers_ok(attr.numRegs)) return cudaErrorLaunchOutOfResources;
  return cudaFuncSetAttribute(attend_kernel<F8>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              smem_bytes<F8>());
}

// What the launches of a cache need, once a device: one cache's kernel that cannot run does not
// turn off the other's.
template <bool F8>
cudaError_t prepare() {
  static std::atomic<int> done[KT_MAX_DEVICES];
  return (cudaError_t)per_device_cached(done, [] {
    cudaError_t r = prepare_attend<F8>();
    if (r == cudaSuccess)
      r = cudaFuncSetAttribute(combine_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                               (int)combine_smem(1, 1));
    if (r == cudaSuccess)
      r = cudaFuncSetAttribute(plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                               (int)sizeof(PlanShared));
    return (int)r;
  });
}

}  // namespace

size_t prefix_ws_bytes(int B, int H_kv, int G) { return prefix_layout(B, H_kv, G).total; }

cudaError_t launch_prefix(const PrefixLaunch& a, cudaStream_t stream) {
  Params p;
  std::memset(&p, 0, sizeof(p));
  const PrefixWs L = prefix_layout(a.B, a.H_kv, a.G);
  uint8_t* ws = static_cast<uint8_t*>(a.ws);
  p.q = a.q;
  p.kmap = *a.kmap;
  p.vmap = *a.vmap;
  p.table = a.table;
  p.seq_lens = a.seq_lens;
  p.cu = a.cu;
  p.prefix = a.prefix;
  p.out = a.out;
  p.status = a.status;
  p.head = reinterpret_cast<Head*>(ws + L.head);
  p.items_a = reinterpret_cast<Item*>(ws + L.items_a);
  p.items_b = reinterpret_cast<Item*>(ws + L.items_b);
  p.cost_a = reinterpret_cast<int*>(ws + L.cost_a);
  p.cost_b = reinterpret_cast<int*>(ws + L.cost_b);
  p.q_rows = reinterpret_cast<int*>(ws + L.q_rows);
  p.seqs = reinterpret_cast<SeqPlan*>(ws + L.seqs);
  p.parts = reinterpret_cast<float*>(ws + L.parts);
  p.stats = reinterpret_cast<float2*>(ws + L.stats);
  p.rows_a = L.rows_a;
  p.B = a.B;
  p.H_kv = a.H_kv;
  p.G = a.G;
  p.groups = a.groups;
  p.max_blocks = a.max_blocks;
  p.P = a.P;
  p.ctas = a.ctas < PREFIX_MAX_CTAS ? a.ctas : PREFIX_MAX_CTAS;
  p.row_max = a.B * a.G < ROWS ? a.B * a.G : ROWS;
  p.scale_log2 = a.scale_log2;
  p.k_scale = a.k_scale;
  p.v_scale = a.v_scale;
  cudaError_t e = a.k_scale ? prepare<true>() : prepare<false>();
  if (e != cudaSuccess) return e;
  int threads = a.B > a.groups + 1 ? a.B : a.groups + 1;
  threads = threads < 64 ? 64 : threads < PLAN_THREADS ? (threads + 31) & ~31 : PLAN_THREADS;
  e = launch(plan_kernel, p, 1, threads, sizeof(PlanShared), stream);
  if (e != cudaSuccess) return e;
  e = a.k_scale ? launch(attend_kernel<true>, p, p.ctas, Config<true>::threads, smem_bytes<true>(),
                         stream)
                : launch(attend_kernel<false>, p, p.ctas, Config<false>::threads, smem_bytes<false>(),
                         stream);
  if (e != cudaSuccess) return e;
  const int jobs = a.H_kv * ((a.B * a.G + COMBINE_ROWS - 1) / COMBINE_ROWS) * (D / 16);
  const int grid = (jobs + COMBINE_WARPS - 1) / COMBINE_WARPS;
  return launch(combine_kernel, p, grid, COMBINE_WARPS * 32, combine_smem(grid, p.ctas), stream);
}

}  // namespace kt
