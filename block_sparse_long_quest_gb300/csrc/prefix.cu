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
//   combine  a warp a row.
#include <cstring>

#include "kt_internal.cuh"

namespace kt {
namespace {

constexpr int ROWS = 128;                // rows of a tile: the M of the tensor-core steps
constexpr int SLOTS = 2;                 // tiles (each with its own scores and output) a CTA
constexpr int SOFT_WARPS = 16;           // two threads a row
constexpr int THREADS = (SOFT_WARPS + 4) * 32;
constexpr int BOX = BS * 64 * 2;         // 128 tokens (or rows) x 64 channels, binary16
constexpr int TILE = 2 * BOX;            // 128 x 128
constexpr int ENTRIES = 5;               // K or V tiles in the ring
constexpr int PLAN_THREADS = 1024;

struct Item {      // blocks of one K/V head that a set of rows attends, for every K/V head
  int seq;         // whose table row to read
  int start;       // first block
  int blocks;
  int rows;        // B items: at most ROWS; A items (two tiles): at most 2 * ROWS
  int member;      // first row's place in the list of members times G, -1: seq's own rows
  int tokens;      // tokens of seq from block `start` on
  int row_base;    // B items: first row of the item's parts (head 0)
  int cum;         // steps of all items before (all heads)
};

struct Start {     // where a CTA (A) or a slot (B; slot s of CTA c is worker s * CTAs + c) begins
  int item, head, block, steps;
};

struct RowPlan {   // where the parts of a row's prefix are
  int kind;        // 0 none, 1 A item, 2 B item
  int item, row, pad;
};

struct Head {
  int steps_a, steps_b, items_b, pad;
};

// Offsets in the workspace's part.
struct PrefixWs {
  size_t head, items_a, items_b, start_a, start_b, members, rows, suffix, parts, stats, total;
  long long rows_a;  // parts of A items come first
};

struct Params {
  CUtensorMap kmap, vmap;
  const __half* q;
  const int32_t* table;
  const int32_t* seq_lens;
  const int32_t* cu;
  const int32_t* prefix;
  float* out;
  int* status;
  Head* head;
  Item* items_a;
  Item* items_b;
  Start* start_a;
  Start* start_b;
  int* members;
  RowPlan* rows;   // [B][G]
  int* suffix;     // [B]: the B item of a sequence's own blocks
  float* parts;    // [rows][128]
  float* stats;    // [rows][4]: m, l of the first and second 64 tokens of each block
  long long rows_a;
  int B, H_kv, G, groups, max_blocks, P, ctas, row_max;
  float scale_log2;
};

__device__ __forceinline__ float ex2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// ---- plan --------------------------------------------------------------------------------
struct PlanShared {
  int cu[MAX_SEGS + 1];
  int member[MAX_SEGS + 1];     // members before sequence b (each in its group)
  int start[MAX_SEGS];          // first block of its own, -1: no member
  int cum_b[2 * MAX_SEGS + 1];
  int cum_a[MAX_SEGS + 1];
  int warp_sum[PLAN_THREADS / 32];
  int bad;
};

__device__ __forceinline__ int plan_scan(int x, int* total, PlanShared& sh) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int incl = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += v;
  }
  __syncthreads();
  if (lane == 31) sh.warp_sum[warp] = incl;
  __syncthreads();
  int s = sh.warp_sum[lane];
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, s, o);
    if (lane >= o) s += v;
  }
  *total = __shfl_sync(0xffffffffu, s, 31);
  const int before = __shfl_sync(0xffffffffu, s, warp > 0 ? warp - 1 : 0);
  return (warp > 0 ? before : 0) + incl - x;
}

// The last index i of [0, n) with cum[i] <= x.
__device__ __forceinline__ int last_at(const int* cum, int n, int x) {
  int lo = 0, hi = n;
  while (lo + 1 < hi) {
    const int mid = (lo + hi) / 2;
    if (cum[mid] <= x) lo = mid;
    else hi = mid;
  }
  return lo;
}

// Workers among whom `all` steps are shared out: each gets at least one.
__device__ __forceinline__ int workers(int n, int all) { return min(n, all); }

__device__ __forceinline__ int seq_len(const Params& p, int b) {
  int n = p.seq_lens[b];
  if (n < 0 || n > p.max_blocks * BS) {
    set_status(p.status, KT_ERR_DEVICE_CHECK);
    n = n < 0 ? 0 : p.max_blocks * BS;
  }
  return n;
}

__global__ void __launch_bounds__(PLAN_THREADS) plan_kernel(const __grid_constant__ Params p) {
  extern __shared__ uint8_t plan_smem[];
  PlanShared& sh = *reinterpret_cast<PlanShared*>(plan_smem);
  griddep_wait();
  griddep_launch_dependents();
  const int tid = threadIdx.x;
  if (tid == 0) sh.bad = 0;
  __syncthreads();
  for (int g = tid; g <= p.groups; g += PLAN_THREADS) {
    const int c = p.cu[g];
    sh.cu[g] = c;
    if (c < 0 || c > p.B || (g > 0 && c < p.cu[g - 1])) sh.bad = 1;
  }
  __syncthreads();
  const bool grouped = !sh.bad;  // else every sequence is attended by itself
  if (!grouped && tid == 0) set_status(p.status, KT_ERR_DEVICE_CHECK);

  // members: sequences that hold all blocks of their group's prefix
  int members = 0;
  for (int b0 = 0; b0 < p.B; b0 += PLAN_THREADS) {
    const int b = b0 + tid;
    int start = -1;
    if (b < p.B && grouped) {
      const int g = last_at(sh.cu, p.groups + 1, b);
      if (g < p.groups && sh.cu[g] <= b) {
        const int blocks = p.prefix[g];
        if (blocks < 0 || blocks > p.max_blocks) set_status(p.status, KT_ERR_DEVICE_CHECK);
        else if (blocks > 0 && seq_len(p, b) >= blocks * BS) start = blocks;
      }
    }
    int total;
    const int r = members + plan_scan(start >= 0, &total, sh);
    if (b < p.B) {
      sh.start[b] = start;
      sh.member[b] = r;
      if (start >= 0) p.members[r] = b;
    }
    members += total;
  }
  if (tid == 0) sh.member[p.B] = members;
  __syncthreads();

  // groups: rows in tiles of 128, two at a time (A items), a last single one a B item
  int pairs = 0, singles = 0, steps_a = 0, steps_b = 0, rows_b = 0;
  for (int g0 = 0; g0 < (grouped ? p.groups : 0); g0 += PLAN_THREADS) {
    const int g = g0 + tid;
    int rows = 0, first = 0, blocks = 0;
    if (g < p.groups) {
      first = sh.member[sh.cu[g]];
      const int n = sh.member[sh.cu[g + 1]] - first;
      if (n >= 2) {
        rows = n * p.G;
        blocks = p.prefix[g];
      }
    }
    const int tiles = (rows + ROWS - 1) / ROWS, np = tiles / 2, ns = tiles & 1;
    const int left = ns ? rows - np * 2 * ROWS : 0;
    int tp, ts, ta, tb, tr;
    const int ip = pairs + plan_scan(np, &tp, sh);
    const int is = singles + plan_scan(ns, &ts, sh);
    const int sa = steps_a + plan_scan(np * blocks, &ta, sh);
    const int sb = steps_b + plan_scan(ns * blocks, &tb, sh);
    const int rb = rows_b + plan_scan(left, &tr, sh);
    for (int i = 0; i < np; ++i) {
      Item it;
      it.seq = p.members[first];
      it.start = 0;
      it.blocks = blocks;
      it.rows = min(2 * ROWS, rows - i * 2 * ROWS);
      it.member = first * p.G + i * 2 * ROWS;
      it.tokens = blocks * BS;
      it.row_base = 0;
      it.cum = (sa + i * blocks) * p.H_kv;
      p.items_a[ip + i] = it;
      sh.cum_a[ip + i] = it.cum;
    }
    if (ns) {
      Item it;
      it.seq = p.members[first];
      it.start = 0;
      it.blocks = blocks;
      it.rows = left;
      it.member = first * p.G + np * 2 * ROWS;
      it.tokens = blocks * BS;
      it.row_base = rb * p.H_kv;
      it.cum = sb * p.H_kv;
      p.items_b[is] = it;
      sh.cum_b[is] = it.cum;
    }
    // where the rows of the group's members find their parts
    for (int r = 0; r < rows; ++r) {
      RowPlan rp;
      const int t = r / ROWS;
      rp.kind = t < 2 * np ? 1 : 2;
      rp.item = t < 2 * np ? ip + t / 2 : is;
      rp.row = t < 2 * np ? r % (2 * ROWS) : r - np * 2 * ROWS;
      rp.pad = 0;
      p.rows[(size_t)p.members[first + r / p.G] * p.G + r % p.G] = rp;
    }
    pairs += tp;
    singles += ts;
    steps_a += ta;
    steps_b += tb;
    rows_b += tr;
  }
  __syncthreads();

  // what each sequence has of its own
  for (int b0 = 0; b0 < p.B; b0 += PLAN_THREADS) {
    const int b = b0 + tid;
    int start = 0, n = 0, nb = 0;
    if (b < p.B) {
      n = seq_len(p, b);
      nb = (n + BS - 1) / BS;
      if (sh.start[b] >= 0) {
        const int g = last_at(sh.cu, p.groups + 1, b);
        if (sh.member[sh.cu[g + 1]] - sh.member[sh.cu[g]] >= 2) start = sh.start[b];
      }
      if (start == 0)
        for (int r = 0; r < p.G; ++r) p.rows[(size_t)b * p.G + r] = RowPlan{0, 0, 0, 0};
    }
    int total;
    const int sb = steps_b + plan_scan(nb - start, &total, sh);
    if (b < p.B) {
      Item it;
      it.seq = b;
      it.start = start;
      it.blocks = nb - start;
      it.rows = p.G;
      it.member = -1;
      it.tokens = n - start * BS;
      it.row_base = (rows_b + b * p.G) * p.H_kv;
      it.cum = sb * p.H_kv;
      p.items_b[singles + b] = it;
      sh.cum_b[singles + b] = it.cum;
      p.suffix[b] = singles + b;
    }
    steps_b += total;
  }
  __syncthreads();
  steps_a *= p.H_kv;
  steps_b *= p.H_kv;
  const int items_b = singles + p.B;
  if (tid == 0) *p.head = Head{steps_a, steps_b, items_b, 0};
  // equal shares: A steps over the CTAs, B steps over their slots
  for (int c = tid; c < p.ctas * (1 + SLOTS); c += PLAN_THREADS) {
    const bool a = c < p.ctas;
    const int w = a ? c : c - p.ctas;
    const long long all = a ? steps_a : steps_b;
    const int n = workers(a ? p.ctas : p.ctas * SLOTS, (int)all);
    Start st = {0, 0, 0, 0};
    if (w < n) {
      const int lo = (int)(all * w / n);
      st.steps = (int)(all * (w + 1) / n) - lo;
      const int* cum = a ? sh.cum_a : sh.cum_b;
      st.item = last_at(cum, a ? pairs : items_b, lo);  // never one without blocks
      const int next = st.item + 1 < (a ? pairs : items_b) ? cum[st.item + 1] : (int)all;
      const int blocks = (next - cum[st.item]) / p.H_kv;
      st.head = (lo - cum[st.item]) / blocks;
      st.block = (lo - cum[st.item]) % blocks;
    }
    (a ? p.start_a : p.start_b)[w] = st;
  }
}

// ---- attend ------------------------------------------------------------------------------
// Warps 0-15 hold the rows: warp w has slot w / 8, the 32 TMEM lanes of quarter w % 4 and
// half (w / 4) % 2 of the columns, so a row's 128 scores and 128 output channels are two
// threads'.  Warps 16 and 17 issue the tensor-core steps of a slot each, so that one slot's
// fill the pauses of the other's; warp 18 loads K and V tiles into a ring of 32 KB entries.
//
// A slot's block: S (TMEM, 128 columns) = Q K^T; the row threads turn it into P, which takes
// the place of S; O (128 columns) = P V; the row threads add it to their running output in
// registers: out = out * 2^(m_old - m_new) + O.  So a block's P V is summed apart from the
// running output, and no output is rescaled in TMEM.
//
// P is held as two binary16, 2^15 p = hi + lo (22 bits, exact to 2^-24 of the largest), and
// P V as two products: with one alone the output would be good to 11 bits only, and it is
// binary32.  For 16 tokens, the K of a tensor-core step, columns 0-7 are hi, 8-15 lo.
//
// A items (two tiles of rows over the same blocks) go through both slots at once, each K/V
// tile read once; with B items the slots are on their own, each with its own share.
struct Misc {
  uint64_t full[ENTRIES], empty[ENTRIES];
  uint64_t s_full[SLOTS], p_full[SLOTS], o_full[SLOTS], q_full[SLOTS];
  uint32_t tmem;
  int bad[ENTRIES];              // the entry's page is outside the pool
  float most[SLOTS][2][ROWS];    // a row's two halves' maxima
};
constexpr int SMEM = SLOTS * TILE + ENTRIES * TILE + sizeof(Misc);
static_assert(SMEM <= 232448, "shared memory of a CTA");
static_assert(SMEM > 233472 / 2, "one CTA an SM: it holds all of TMEM");
constexpr uint32_t TMEM_COLS = 512;

// 16 columns of this thread's TMEM lane to and from registers.
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, float (&v)[16]) {
  uint32_t r[16];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,"
      "%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r[i]);
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

// Scores of tokens from `valid` on leave the softmax; v holds those of tokens first ...
__device__ __forceinline__ void mask16(float (&v)[16], int first, int valid) {
#pragma unroll
  for (int j = 0; j < 16; ++j)
    if (first + j >= valid) v[j] = -INFINITY;
}

// Registers pass from the control warps to the row threads: five warpgroups are launched with
// LAUNCH_REGS a thread (the host checks that), and the shares must not add up to more.
constexpr int LAUNCH_REGS = 96, ROW_REGS = 104, CONTROL_REGS = 64;
static_assert(4 * ROW_REGS + CONTROL_REGS <= 5 * LAUNCH_REGS, "registers of a CTA");
template <int N>
__device__ __forceinline__ void regs_inc() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void regs_dec() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

// A walk over the steps of a share: runs of blocks of one (item, head).
struct Walk {
  const Item* items;
  int item, head, block, left;  // `left` steps of the share
};
__device__ __forceinline__ Walk walk_of(const Item* items, const Start& s) {
  return Walk{items, s.item, s.head, s.block, s.steps};
}
// The run at the walk's place; call advance(run) afterwards.
__device__ __forceinline__ int run_of(const Walk& w, const Item& it) {
  return min(w.left, it.blocks - w.block);
}
__device__ __forceinline__ void advance(Walk& w, int run, int heads) {
  w.left -= run;
  w.block = 0;
  if (++w.head == heads) {
    w.head = 0;
    ++w.item;
    while (w.left > 0 && w.items[w.item].blocks == 0) ++w.item;
  }
}

// First ring entry of slot s's B step k (K; V is the next one), behind `a` A steps: the
// slots' steps take turns as long as both have some.
__device__ __forceinline__ int entry_b(int s, int k, int a, int other) {
  return 2 * (a + k + min(s == 0 ? k : k + 1, other));
}

__device__ __forceinline__ uint32_t entry_parity(int e) { return (uint32_t)(e / ENTRIES) & 1u; }

__global__ void __launch_bounds__(THREADS, 1) attend_kernel(const __grid_constant__ Params p) {
  extern __shared__ __align__(1024) uint8_t smem[];
  Misc& ms = *reinterpret_cast<Misc*>(smem + (SLOTS + ENTRIES) * TILE);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int cta = blockIdx.x;
  const uint32_t sQ = smem_u32(smem), ring = sQ + SLOTS * TILE;
  const uint32_t full = smem_u32(ms.full), empty = smem_u32(ms.empty);
  const uint32_t s_full = smem_u32(ms.s_full), p_full = smem_u32(ms.p_full);
  const uint32_t o_full = smem_u32(ms.o_full), q_full = smem_u32(ms.q_full);
  if (tid == 0) {
    for (int i = 0; i < ENTRIES; ++i) {
      mbar_init(full + 8 * i, 1);
      mbar_init(empty + 8 * i, 2);
    }
    for (int i = 0; i < SLOTS; ++i) {
      mbar_init(s_full + 8 * i, 1);
      mbar_init(p_full + 8 * i, SOFT_WARPS / SLOTS);
      mbar_init(o_full + 8 * i, 1);
      mbar_init(q_full + 8 * i, SOFT_WARPS / SLOTS);
    }
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
  const Start sa = p.start_a[cta];
  const Start sb0 = p.start_b[cta], sb1 = p.start_b[p.ctas + cta];

  if (warp < SOFT_WARPS) regs_inc<ROW_REGS>();
  else regs_dec<CONTROL_REGS>();
  if (warp == SOFT_WARPS + 2) {
    // ============================ K and V tiles ============================
    if (lane == 0) {
      const uint64_t pol = l2_evict_first_policy();
      const int row_end = p.P * p.H_kv * BS;  // reads zeros
      int e = 0;
      bool ok = true;
      auto load = [&](const Item& it, int head, int block) {
        const int page = p.table[(size_t)it.seq * p.max_blocks + it.start + block];
        const bool bad = page < 0 || page >= p.P;
        if (bad) set_status(p.status, KT_ERR_DEVICE_CHECK);
        const int row = bad ? row_end : (page * p.H_kv + head) * BS;
        for (int side = 0; side < 2; ++side, ++e) {
          const int st = e % ENTRIES;
          if (e >= ENTRIES && !mbar_wait(empty + 8 * st, entry_parity(e) ^ 1, p.status)) return false;
          const CUtensorMap* map = side == 0 ? &p.kmap : &p.vmap;
          const uint32_t dst = ring + st * TILE;
          ms.bad[st] = bad;
          mbar_arrive_expect_tx(full + 8 * st, TILE);
          tma_load_2d(dst, map, 0, row, full + 8 * st, pol);
          tma_load_2d(dst + BOX, map, 64, row, full + 8 * st, pol);
        }
        return true;
      };
      Walk w = walk_of(p.items_a, sa);
      while (ok && w.left > 0) {
        const Item it = w.items[w.item];
        const int run = run_of(w, it);
        for (int i = 0; i < run && ok; ++i) ok = load(it, w.head, w.block + i);
        advance(w, run, p.H_kv);
      }
      Walk ws[SLOTS] = {walk_of(p.items_b, sb0), walk_of(p.items_b, sb1)};
      while (ok && (ws[0].left > 0 || ws[1].left > 0)) {
#pragma unroll
        for (int s = 0; s < SLOTS; ++s) {
          Walk& x = ws[s];
          if (x.left > 0 && ok) {
            const Item it = x.items[x.item];
            ok = load(it, x.head, x.block);
            if (x.block + 1 < it.blocks) {
              --x.left;
              ++x.block;
            } else {
              advance(x, 1, p.H_kv);
            }
          }
        }
      }
      // nothing of this CTA's is in flight when it ends
      for (int i = max(0, e - ENTRIES); i < e; ++i)
        mbar_wait(full + 8 * (i % ENTRIES), entry_parity(i), p.status);
    }
    __syncwarp();
  } else if (warp == SOFT_WARPS || warp == SOFT_WARPS + 1) {
    // ============================ tensor-core steps ============================
    if (lane == 0) {
      const int s = warp - SOFT_WARPS;
      const uint32_t q = sQ + s * TILE, st = tmem + s * 256, ot = st + 128;
      const int other = s == 0 ? sb1.steps : sb0.steps;
      int k = 0, units = 0;
      bool ok = true;
      for (int part = 0; part < 2 && ok; ++part) {
        const bool a = part == 0;
        Walk w = a ? walk_of(p.items_a, sa) : walk_of(p.items_b, s == 0 ? sb0 : sb1);
        while (ok && w.left > 0) {
          const int run = min(w.left, w.items[w.item].blocks - w.block);
          for (int i = 0; i < run && ok; ++i, ++k) {
            const int e = a ? 2 * k : entry_b(s, k - sa.steps, sa.steps, other);
            const int ek = e % ENTRIES, ev = (e + 1) % ENTRIES;
            // S = Q K^T once K, the run's Q and the end of the last P V are there
            ok = mbar_wait(full + 8 * ek, entry_parity(e), p.status) &&
                 (i > 0 || mbar_wait(q_full + 8 * s, units & 1, p.status)) &&
                 (k == 0 || mbar_wait(o_full + 8 * s, (k - 1) & 1, p.status));
            if (!ok) break;
            tc_fence_after();
            const uint32_t kb = ring + ek * TILE;
#pragma unroll
            for (int ks = 0; ks < 8; ++ks)
              umma_f16(st, umma_sdesc_sw128(q + (ks >> 2) * BOX + (ks & 3) * 32),
                       umma_sdesc_sw128(kb + (ks >> 2) * BOX + (ks & 3) * 32), IDESC_S, ks > 0);
            umma_commit(s_full + 8 * s);
            umma_commit(empty + 8 * ek);
            if (!a) umma_commit(empty + 8 * ek);  // the other slot has no part in this one
            // O = P V, the high and the low parts of P
            ok = mbar_wait(full + 8 * ev, entry_parity(e + 1), p.status) &&
                 mbar_wait(p_full + 8 * s, k & 1, p.status);
            if (!ok) break;
            tc_fence_after();
            const uint32_t vb = ring + ev * TILE;
#pragma unroll
            for (int ks = 0; ks < 16; ++ks)
              umma_f16_ta(ot, st + (ks & 7) * 16 + (ks >> 3) * 8,
                          sdesc_mn_sw128(vb + (ks & 7) * 2048), IDESC_O, ks > 0);
            umma_commit(o_full + 8 * s);
            umma_commit(empty + 8 * ev);
            if (!a) umma_commit(empty + 8 * ev);
          }
          ++units;
          advance(w, run, p.H_kv);
        }
      }
    }
    __syncwarp();
  } else if (warp < SOFT_WARPS) {
    // ============================ rows ============================
    const int s = warp >> 3, quarter = warp & 3, half = (warp >> 2) & 1;
    const int r = quarter * 32 + lane;       // this thread's row
    const int st_tid = tid & 255;
    const uint32_t tb = tmem + s * 256 + ((uint32_t)(quarter * 32) << 16) + half * 64;
    const int H_q = p.H_kv * p.G;
    const Start sb = s == 0 ? sb0 : sb1;
    const int other = s == 0 ? sb1.steps : sb0.steps;
    int k = 0;
    bool ok = true;
    for (int part = 0; part < 2 && ok; ++part) {
      const bool a = part == 0;
      Walk w = a ? walk_of(p.items_a, sa) : walk_of(p.items_b, sb);
      while (w.left > 0 && ok) {
        const Item it = w.items[w.item];
        const int run = run_of(w, it);
        const int off = a ? s * ROWS : 0;    // the slot's tile of an A item
        const int rows = min(ROWS, it.rows - off);
        // queries into two swizzled boxes (chunk c of row i: box c / 8, slot (c % 8) ^ (i % 8))
        uint8_t* q = smem + s * TILE;
        for (int idx = st_tid; idx < rows * 16; idx += 256) {
          const int i = idx >> 4, c = idx & 15;
          int b = it.seq, g = i;
          if (it.member >= 0) {
            const int m = it.member + off + i;
            b = p.members[m / p.G];
            g = m % p.G;
          }
          const uint4 v = *(reinterpret_cast<const uint4*>(
                                p.q + ((size_t)b * H_q + w.head * p.G + g) * D) + c);
          *reinterpret_cast<uint4*>(q + (c >> 3) * BOX + i * 128 + (((c & 7) ^ (i & 7)) << 4)) = v;
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(q_full + 8 * s);

        const bool active = quarter * 32 < rows;
        float acc[64], m = -INFINITY, l = 0.0f;
#pragma unroll
        for (int i = 0; i < 64; ++i) acc[i] = 0.0f;
        for (int i = 0; i < run && ok; ++i, ++k) {
          const int e = (a ? 2 * k : entry_b(s, k - sa.steps, sa.steps, other)) + 1;  // V's entry
          const int ev = e % ENTRIES;
          ok = mbar_wait(s_full + 8 * s, k & 1, p.status);
          if (!ok) break;
          tc_fence_after();
          int valid = min(BS, it.tokens - (w.block + i) * BS);
          if (valid < BS) {
            // V behind the last token may be anything, and 0 * NaN is NaN: zeros there
            ok = mbar_wait(full + 8 * ev, entry_parity(e), p.status);
            if (!ok) break;
            uint8_t* v = smem + SLOTS * TILE + ev * TILE;
            for (int idx = valid * 8 + st_tid; idx < BS * 8; idx += 256) {
              *reinterpret_cast<uint4*>(v + idx * 16) = make_uint4(0, 0, 0, 0);
              *reinterpret_cast<uint4*>(v + BOX + idx * 16) = make_uint4(0, 0, 0, 0);
            }
            fence_proxy_async_smem();
          }
          float alpha = 1.0f;
          if (active) {
            if (!mbar_try_wait(full + 8 * ev, entry_parity(e)))
              ok = mbar_wait(full + 8 * ev, entry_parity(e), p.status);
            if (ms.bad[ev]) valid = 0;
            float mx = -INFINITY;
#pragma unroll
            for (int c = 0; c < 64; c += 16) {
              float v[16];
              tmem_ld16(tb + c, v);
              if (valid < BS) mask16(v, half * 64 + c, valid);
              float m4[4] = {v[0], v[1], v[2], v[3]};
#pragma unroll
              for (int j = 4; j < 16; ++j) m4[j & 3] = fmaxf(m4[j & 3], v[j]);
              mx = fmaxf(mx, fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3])));
            }
            ms.most[s][half][r] = mx;
            named_bar_sync(1 + s * 4 + quarter, 64);
            mx = fmaxf(mx, ms.most[s][half ^ 1][r]);
            const float m_new = fmaxf(m, mx * p.scale_log2);
            const float base = m_new == -INFINITY ? 0.0f : m_new;
            alpha = ex2_fast(m - base);
            m = m_new;
            const float shift = 15.0f - base;
            float sum4[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int c = 0; c < 64; c += 16) {
              float v[16];
              uint32_t w16[16];
              tmem_ld16(tb + c, v);
              if (valid < BS) mask16(v, half * 64 + c, valid);
#pragma unroll
              for (int j = 0; j < 16; j += 2) {
                const float x = ex2_fast(fmaf(v[j], p.scale_log2, shift));
                const float y = ex2_fast(fmaf(v[j + 1], p.scale_log2, shift));
                sum4[j & 3] += x;
                sum4[(j & 3) + 1] += y;
                const __half2 hi = __floats2half2_rn(x, y);
                const float2 back = __half22float2(hi);
                const __half2 lo = __floats2half2_rn(x - back.x, y - back.y);
                w16[j / 2] = *reinterpret_cast<const uint32_t*>(&hi);
                w16[8 + j / 2] = *reinterpret_cast<const uint32_t*>(&lo);
              }
              tmem_st16(tb + c, w16);
            }
            l = fmaf(l, alpha, (sum4[0] + sum4[1]) + (sum4[2] + sum4[3]));
            tmem_wait_st();
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(p_full + 8 * s);
          ok = mbar_wait(o_full + 8 * s, k & 1, p.status) && ok;
          if (!ok) break;
          tc_fence_after();
          if (active) {
#pragma unroll
            for (int c = 0; c < 64; c += 16) {
              float v[16];
              tmem_ld16(tb + 128 + c, v);
#pragma unroll
              for (int j = 0; j < 16; ++j) acc[c + j] = fmaf(acc[c + j], alpha, v[j]);
            }
          }
        }
        // this run's part of the rows
        if (r < rows && ok) {
          const size_t row =
              a ? ((size_t)cta + (size_t)w.item * p.H_kv + w.head) * (2 * ROWS) + off + r
                : (size_t)p.rows_a + (size_t)(s * p.ctas + cta) * p.row_max + it.row_base +
                      (size_t)w.head * it.rows + r;
          float4* o = reinterpret_cast<float4*>(p.parts + row * D + half * 64);
#pragma unroll
          for (int i = 0; i < 16; ++i)
            o[i] = make_float4(acc[4 * i], acc[4 * i + 1], acc[4 * i + 2], acc[4 * i + 3]);
          if (half == 0) p.stats[row * 4] = m;
          p.stats[row * 4 + 1 + half] = l;
        }
        advance(w, run, p.H_kv);
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
constexpr int COMBINE_WARPS = 8;

// The worker of `n` with equal shares of `all` steps that takes step x.
__device__ __forceinline__ int worker_of(int x, int all, int n) {
  int w = (int)((long long)x * n / all);
  while (w + 1 < n && (long long)all * (w + 1) / n <= x) ++w;
  while (w > 0 && (long long)all * w / n > x) --w;
  return w;
}

__global__ void __launch_bounds__(COMBINE_WARPS * 32) combine_kernel(const __grid_constant__ Params p) {
  griddep_wait();
  griddep_launch_dependents();
  const int lane = threadIdx.x & 31;
  const int H_q = p.H_kv * p.G;
  const int row = blockIdx.x * COMBINE_WARPS + (threadIdx.x >> 5);
  if (row >= p.B * H_q) return;
  const int b = row / H_q, hq = row % H_q, h = hq / p.G, g = hq % p.G;
  const Head head = *p.head;
  const RowPlan rp = p.rows[(size_t)b * p.G + g];
  const Item own = p.items_b[p.suffix[b]];
  // parts: of the prefix, then of the sequence's own blocks; place i is a + i * stride
  size_t at[2] = {0, 0};
  size_t stride[2] = {0, 0};
  int n[2] = {0, 0};
  const int workers_a = workers(p.ctas, head.steps_a);
  const int workers_b = workers(p.ctas * SLOTS, head.steps_b);
  if (rp.kind == 1) {
    const Item it = p.items_a[rp.item];
    const int x = it.cum + h * it.blocks;
    const int c0 = worker_of(x, head.steps_a, workers_a);
    n[0] = worker_of(x + it.blocks - 1, head.steps_a, workers_a) - c0 + 1;
    at[0] = ((size_t)c0 + (size_t)rp.item * p.H_kv + h) * (2 * ROWS) + rp.row;
    stride[0] = 2 * ROWS;
  } else if (rp.kind == 2) {
    const Item it = p.items_b[rp.item];
    const int x = it.cum + h * it.blocks;
    const int c0 = worker_of(x, head.steps_b, workers_b);
    n[0] = worker_of(x + it.blocks - 1, head.steps_b, workers_b) - c0 + 1;
    at[0] = (size_t)p.rows_a + (size_t)c0 * p.row_max + it.row_base + (size_t)h * it.rows + rp.row;
    stride[0] = p.row_max;
  }
  if (own.blocks > 0) {
    const int x = own.cum + h * own.blocks;
    const int c0 = worker_of(x, head.steps_b, workers_b);
    n[1] = worker_of(x + own.blocks - 1, head.steps_b, workers_b) - c0 + 1;
    at[1] = (size_t)p.rows_a + (size_t)c0 * p.row_max + own.row_base + (size_t)h * own.rows + g;
    stride[1] = p.row_max;
  }
  float M = -INFINITY;
  for (int k = 0; k < 2; ++k)
    for (int i = lane; i < n[k]; i += 32) M = fmaxf(M, p.stats[(at[k] + i * stride[k]) * 4]);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
  const float base = M == -INFINITY ? 0.0f : M;
  float L = 0.0f;
  float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  for (int k = 0; k < 2; ++k)
#pragma unroll 4
    for (int i = 0; i < n[k]; ++i) {
      const size_t r = at[k] + i * stride[k];
      const float4 st = *reinterpret_cast<const float4*>(p.stats + r * 4);
      const float4 o = *reinterpret_cast<const float4*>(p.parts + r * D + lane * 4);
      const float w = ex2_fast(st.x - base);
      L = fmaf(st.y + st.z, w, L);
      acc.x = fmaf(o.x, w, acc.x);
      acc.y = fmaf(o.y, w, acc.y);
      acc.z = fmaf(o.z, w, acc.z);
      acc.w = fmaf(o.w, w, acc.w);
    }
  const float inv = L == 0.0f ? 0.0f : 1.0f / L;
  reinterpret_cast<float4*>(p.out + (size_t)row * D)[lane] =
      make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv);
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
  L.start_a = off;
  off = align256(off + PREFIX_MAX_CTAS * sizeof(Start));
  L.start_b = off;
  off = align256(off + PREFIX_MAX_CTAS * SLOTS * sizeof(Start));
  L.members = off;
  off = align256(off + (size_t)B * 4);
  L.rows = off;
  off = align256(off + (size_t)B * G * sizeof(RowPlan));
  L.suffix = off;
  off = align256(off + (size_t)B * 4);
  // A items: 256 rows for each (CTA, item and head) that meet; there are fewer than CTAs +
  // items of those.  B items: row_max rows a slot and the rows of all items.
  L.rows_a = B * G > ROWS ? (long long)(PREFIX_MAX_CTAS + max_pairs * H_kv) * 2 * ROWS : 0;
  const size_t total_rows = L.rows_a + (size_t)PREFIX_MAX_CTAS * SLOTS * row_max + 2 * rows;
  L.parts = off;
  off = align256(off + total_rows * D * 4);
  L.stats = off;
  off = align256(off + total_rows * 16);
  L.total = off + 256;  // (its start is aligned down)
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

}  // namespace

size_t prefix_ws_bytes(int B, int H_kv, int G) { return prefix_layout(B, H_kv, G).total; }

cudaError_t launch_prefix(const PrefixLaunch& a, cudaStream_t stream) {
  Params p;
  std::memset(&p, 0, sizeof(p));
  const PrefixWs L = prefix_layout(a.B, a.H_kv, a.G);
  uint8_t* ws = static_cast<uint8_t*>(a.ws);
  p.kmap = *a.kmap;
  p.vmap = *a.vmap;
  p.q = a.q;
  p.table = a.table;
  p.seq_lens = a.seq_lens;
  p.cu = a.cu;
  p.prefix = a.prefix;
  p.out = a.out;
  p.status = a.status;
  p.head = reinterpret_cast<Head*>(ws + L.head);
  p.items_a = reinterpret_cast<Item*>(ws + L.items_a);
  p.items_b = reinterpret_cast<Item*>(ws + L.items_b);
  p.start_a = reinterpret_cast<Start*>(ws + L.start_a);
  p.start_b = reinterpret_cast<Start*>(ws + L.start_b);
  p.members = reinterpret_cast<int*>(ws + L.members);
  p.rows = reinterpret_cast<RowPlan*>(ws + L.rows);
  p.suffix = reinterpret_cast<int*>(ws + L.suffix);
  p.parts = reinterpret_cast<float*>(ws + L.parts);
  p.stats = reinterpret_cast<float*>(ws + L.stats);
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
  static std::atomic<int> optin[KT_MAX_DEVICES];
  cudaError_t e = (cudaError_t)per_device_cached(optin, [] {
    cudaFuncAttributes attr;
    cudaError_t r = cudaFuncGetAttributes(&attr, attend_kernel);
    if (r != cudaSuccess) return (int)r;
    if (attr.numRegs != LAUNCH_REGS) return (int)cudaErrorLaunchOutOfResources;
    r = cudaFuncSetAttribute(attend_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM);
    if (r != cudaSuccess) return (int)r;
    return (int)cudaFuncSetAttribute(plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                     (int)sizeof(PlanShared));
  });
  if (e != cudaSuccess) return e;
  e = launch(plan_kernel, p, 1, PLAN_THREADS, sizeof(PlanShared), stream);
  if (e != cudaSuccess) return e;
  e = launch(attend_kernel, p, p.ctas, THREADS, SMEM, stream);
  if (e != cudaSuccess) return e;
  const int rows = a.B * a.H_kv * a.G;
  return launch(combine_kernel, p, (rows + COMBINE_WARPS - 1) / COMBINE_WARPS, COMBINE_WARPS * 32, 0,
                stream);
}

}  // namespace kt
