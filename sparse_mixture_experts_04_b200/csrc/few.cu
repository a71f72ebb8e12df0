// The whole layer for a few tokens (1..64) in one kernel.
//
// With a handful of tokens the layer is a stream of weights: the experts that
// got a row are read once, and everything else (routing, activations, the
// combine) is small.  One cooperative kernel, one CTA per SM, keeps that stream
// running from the first byte to the last instead of draining it at the ends
// of six launches:
//
//   1. logits    tiles of 4 experts x 4 tokens over the CTAs; with 8-bit
//                weights also the tokens' integers                  grid barrier
//   2. routing   softmax and top-K: up to 8 tokens every CTA for itself, more
//                of them one token per CTA                          grid barrier
//                capacity and slots: every CTA for itself; CTA 0 writes them
//   3. up        h = silu(W_gate x) * (W_up x)                      grid barrier
//   4. down      partial sums of W_down h, FP32                     grid barrier
//   5. combine   y_t = sum of the shared experts + sum_k w_k Expert_k(x_t)
//
// Steps 3 and 4 are cut into units of 16 weight rows (8 gate rows and their 8
// up rows; 16 output channels), whose reduction stays inside the CTA.  A CTA's
// units are one contiguous range of the list (expert, reduction chunk, rows),
// so a unit's tokens are usually in shared memory already.  The weights come
// through a ring of shared-memory stages filled by bulk copies; the copies run
// ahead of the arithmetic across units and across the grid barriers (weights
// depend on no other CTA), so a barrier costs no bandwidth.
//
// Arithmetic: BF16 and 8-bit weights are the M operand of m16n8k16 / m16n8k32
// tensor-core instructions (16 weight rows, 8 tokens).  Two teams of 4 warps
// take a unit each; the warps of a team take 64-byte slices of the reduction in
// turn, and their 16 x 8 sums are added in shared memory in warp order.  The
// tensor cores are nearly idle while experts have up to 8 rows (a stage of 32 KB
// arrives in 1400 cycles and is multiplied in some 500), so the warp-level
// instruction does: its units of 16 weight rows spread evenly over the SMs, where a
// tcgen05 tile takes 128 weight rows at a time.  With more rows per expert the
// products do set the pace, and moe_layer_forward, whose tiles of few tokens have
// 128 weight rows each as the M operand of tcgen05, is the faster (d = 4096, E = 8,
// F = 14336, top-2: 16 tokens 471 / 430 us, 32 tokens 474 / 574, 64 tokens
// 479 / 853, forward / this kernel).  FP32
// weights take fused multiply-adds (8 rows x 8 tokens per lane), which read an
// expert of more than 8 rows once per 8.  Sums are FP32
// or int32; BF16 layers keep a hidden value as the sum of two BF16 (the tensor
// cores' operands, 16 bits in all) and round nothing else before y.  No step
// depends on the order in which CTAs run, so results repeat bit for bit.
//
// What bounds it: the weights' stream.  us per call, and of the measured copy
// bandwidth (6540 GB/s) that the weights alone make up: 32 tokens, d = 4096,
// E = 128, F = 1536, top-8 + 1 shared 654 (0.99); one token, d = 4096, E = 8,
// F = 14336, top-2 125 (0.86); one token, d = 2048, E = 128, F = 1024, top-8 + 4
// shared 45 (0.51).  The last is where the rest shows: 8.5 us until the experts are
// known (logits 3, barrier 2, top-K 2, slots 1), three more grid barriers of 2 us,
// 3 us for the combine, 2 us between two launches.  Code that runs once per call is
// fetched from memory first, so it is short and has one copy: a second inlined call
// of the selection alone cost 3 us.
//
// The first grid barrier is cooperative groups' own, which needs no cleared
// memory; it has no time limit and needs none: all CTAs are resident (cooperative
// launch) and none waits for anything before it.  CTA 0 clears the counters of
// the others in front of it.  Every wait behind it is bounded (mbar_wait,
// few_grid_sync).  A CTA in which one runs out issues no more copies, runs no
// further pass and no combine (what other CTAs were to write may be missing, row
// indices among it), still arrives at every barrier, waits for its copies in
// flight and reports MOE_DEV_WAIT_TIMEOUT.
#include <cooperative_groups.h>
#include <math.h>

#include <mutex>

#include "common.cuh"
#include "internal.h"
#include "quant.cuh"
#include "router_select.cuh"

namespace moe {

namespace cg = cooperative_groups;

// Variants: the weights' type; kFewBF16Many trades half of the ring for a token
// buffer of twice the rows (see few_tiling).
enum { kFewBF16 = 0, kFewF32 = 1, kFewI8 = 2, kFewBF16Many = 3 };

constexpr int kFewWorkers = 256;                 // 8 warps
constexpr int kFewRows = 16;                     // weight rows of a unit
constexpr int kFewStages = 4;
constexpr int kFewBufBytes = 201728;             // ring and token buffer together
constexpr int kFewMaxPairs = kFewMaxTokens * kMaxTopK;
constexpr int kFewRedBytes = 2 * 8 * 2 * 128 * 4;  // [teams][2][8 / teams warps][2 token tiles][16 x 8] sums

struct FewShared {
  uint64_t full[kFewStages];
  uint64_t empty[kFewStages];
  unsigned long long mask[kMaxExperts];   // tokens that chose the expert
  double fp[kMaxExperts];                 // f_e P_e (statistics)
  unsigned long long scan[8];             // warp totals of few_dispatch's prefix sums
  int counts[kMaxExperts];
  int kept[kMaxExperts];
  int seg_off[kMaxExperts + 1];
  int groups[2][kMaxExperts + 1];         // prefix of the experts' token groups: up, down
  uint16_t perm[kFewMaxPairs];            // slot -> t * K + k
  float row_scale[16];                    // 8-bit tokens: scale of each row in the token buffer
  uint64_t never;                         // a barrier that nothing arrives on (test_stall)
  int abort_flag;                         // raised by whoever gave up a wait
  int gave_up;                            // the worker threads' common view of it (few_grid_sync)
};

constexpr int few_smem_bytes() {
  return kFewBufBytes + kFewRedBytes + static_cast<int>(sizeof(FewShared)) + 128;
}
static_assert(few_smem_bytes() <= 227 * 1024, "shared memory of the few-token kernel");

// Shared-memory tiling of a variant.  A copy of less than 2 KB costs as much to
// issue as one of 2 KB, so smaller chunks take more copying warps.
template <int WT>
struct FewTile {
  static constexpr int kChunk = WT == kFewBF16Many ? 1024 : 2048;  // bytes of each row in a stage
  static constexpr int kPitch = kChunk + 16;                       // odd number of 16-byte pieces: no bank conflicts
  static constexpr int kStageBytes = kFewRows * kPitch;
  static constexpr int kTokBytes = kFewBufBytes - kFewStages * kStageBytes;  // 8 (many: 16) rows of 8 KB
  static constexpr int kCopiers = WT == kFewBF16Many ? 4 : 2;  // warps that issue copies, 16 / kCopiers rows each
  static constexpr int kThreads = kFewWorkers + 32 * kCopiers + 32;  // + one warp for the statistics
};

struct FewArgs {
  const void* x;
  const void* w_gate;
  const float* logit_offset;
  const float* sel_bias;
  const int32_t* expert_cap;  // per-expert capacities, or nullptr
  const char* w13;
  const char* w2;
  const char* w13_s;
  const char* w2_s;
  const float* s13;    // 8-bit weights: scales [E, 2F], [E, d], [N_s, 2F], [d]
  const float* s2;
  const float* s13_s;
  const float* s2_s;
  void* y;
  float* logits;
  int32_t* topk_idx;
  float* topk_w;
  int32_t* counts;
  int32_t* kept;
  int32_t* seg_off;
  int32_t* slot_of;
  int32_t* perm;
  float* stats;        // or nullptr
  void* h;             // [T K, F] hidden rows by slot: BF16, or FP32 (FP32 and 8-bit weights)
  void* h_s;           // [T, N_s F]
  int8_t* x_q;         // 8-bit: the tokens' integers [T, d] and scales [T]
  float* x_scale;
  unsigned* amax;      // 8-bit: bits of max|h| by slot, then by token for the shared experts
  float* part;         // [nc][T K][d] partial sums by slot
  float* part_s;       // [N_s nc][T][d]
  unsigned* status;
  unsigned* arrivals;          // [3] CTAs that reached each grid barrier (cleared before the first)
  unsigned long long* psum;    // [E] sum of p, fixed point (statistics; cleared likewise)
  float* lse2;                 // [T] squared logsumexp of each token (statistics)
  int T, d, E, K, Ns, F;
  long long cap;       // -1: no limit
  int given, bias_on_logit, extended;
  float alpha;
  double pscale;
  int spread;          // top-K: one token per CTA instead of every CTA all tokens
  unsigned long long stall_ns;  // abort-path test hook (test_stall), 0 normally
  // tiling (host): token rows per group, reduction chunks of the down product
  int ng_up, ng_down, nc, chunk_bytes;
};

// ------------------------------------------------------------ small helpers
__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(smem_addr(dst)),
      "l"(src), "r"(bytes), "r"(smem_addr(bar))
      : "memory");
}

__device__ __forceinline__ void ldmatrix_x4(uint32_t saddr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(saddr)
               : "memory");
}

__device__ __forceinline__ void mma_16x8(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void mma_16x8(int (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+r"(c[0]), "+r"(c[1]), "+r"(c[2]), "+r"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Grid barrier of the worker threads: the CTA's writes before it are seen by
// every CTA's reads (past L1) after it.  All CTAs are resident and every one
// of them arrives whatever its copies do; the wait is bounded all the same.
// Whether the CTA may go on: false once any wait in it was given up, the same in
// all worker threads (thread 0 decides; a copying warp may raise the flag any time).
__device__ __forceinline__ bool few_grid_sync(unsigned* arrivals, FewShared& s, unsigned long long limit_ns, int tid) {
  named_bar_sync(1, kFewWorkers);
  if (tid == 0) {
    __threadfence();
    atomicAdd(arrivals, 1u);
    const unsigned long long t0 = global_ns();
    volatile int* abort_flag = &s.abort_flag;
    unsigned n;
    for (unsigned i = 1;; ++i) {
      asm volatile("ld.acquire.gpu.u32 %0, [%1];" : "=r"(n) : "l"(arrivals) : "memory");
      if (n >= gridDim.x) break;
      if ((i & 255u) == 0 && (*abort_flag || global_ns() - t0 > limit_ns)) {
        *abort_flag = 1;
        break;
      }
    }
    __threadfence();
    s.gave_up = *abort_flag;
  }
  named_bar_sync(1, kFewWorkers);
  return s.gave_up == 0;
}

__device__ __forceinline__ float silu(float g) { return g / (1.0f + __expf(-g)); }

// The four passes over weights: shared and routed experts, up and down.
enum { kUpShared = 0, kUpRouted = 1, kDownShared = 2, kDownRouted = 3, kPasses = 4 };

// Where the units of one pass lie and which of them are this CTA's.
struct PassRange {
  int first, last;  // units [first, last)
};

// A run of units over the same tokens, decoded: which weights, which tokens.
struct Span {
  const char* w;       // row 0 of the current unit at the start of its reduction
  int64_t hi;          // byte offset from row r < 8 to row r + 8
  int64_t row_bytes;   // distance between rows
  int units;           // units of the span
  int step;            // features (up: 8) or output channels (down: 16) of a unit
  int col, cols;       // first feature / channel of the current unit, and their number in all
  int len;             // bytes of each row in the unit's reduction
  int e;               // expert (routed or shared)
  int row0, n;         // first token row (slot or token) and their number
  int c;               // reduction chunk (down)
};

template <int WT>
struct Few : FewTile<WT> {
  static constexpr int kW = WT == kFewF32 ? 4 : WT == kFewI8 ? 1 : 2;  // bytes of a weight
  // The worker warps work as teams, each on its own unit: while one adds up its
  // warps' sums and stores them, the other multiplies.
  static constexpr int kTeams = WT == kFewF32 ? 1 : 2;
  static constexpr int kTeamWarps = kFewWorkers / 32 / kTeams;
  // BF16: a hidden value is the sum of two BF16, 16 bits in all, each a row of its
  // own in the token buffer (see few_store_unit).
  static constexpr int kParts = kW == 2 ? 2 : 1;
  using Acc = typename std::conditional<WT == kFewI8, int, float>::type;

  const FewArgs& a;
  FewShared& s;
  uint8_t* ring;
  uint8_t* tok;
  int cta, n_cta, nfb, nb;
  int sg_up, sg_down;  // token groups of a shared expert

  __device__ __forceinline__ Few(const FewArgs& a_, FewShared& s_, uint8_t* ring_, uint8_t* tok_)
      : a(a_), s(s_), ring(ring_), tok(tok_), cta(blockIdx.x), n_cta(gridDim.x), nfb(a_.F / 8),
        nb((a_.d + kFewRows - 1) / kFewRows), sg_up((a_.T + a_.ng_up - 1) / a_.ng_up),
        sg_down((a_.T + a_.ng_down - 1) / a_.ng_down) {}

  // rows of the hidden buffer in front of the low parts
  __device__ __forceinline__ int64_t low_rows(bool routed) const { return static_cast<int64_t>(a.T) * (routed ? a.K : a.Ns); }

  // units of a pass (fewer than 2^31: few_supported)
  __device__ __forceinline__ unsigned units(int pass) const {
    const bool up = pass <= kUpRouted;
    const unsigned groups = pass == kUpRouted || pass == kDownRouted
                                ? s.groups[up ? 0 : 1][a.E]
                                : static_cast<unsigned>(a.Ns) * (up ? sg_up : sg_down);
    return groups * static_cast<unsigned>(up ? nfb : a.nc * nb);
  }
  // this CTA's: n / n_cta of them, the first n % n_cta CTAs one more
  __device__ __forceinline__ PassRange range(int pass) const {
    const unsigned n = units(pass), each = n / n_cta, more = n - each * n_cta;
    const unsigned first = cta * each + min(static_cast<unsigned>(cta), more);
    return PassRange{static_cast<int>(first), static_cast<int>(first + each + (cta < static_cast<int>(more) ? 1 : 0))};
  }

  // expert of routed token group v: the last e with groups[e] <= v, by counting
  // (whole warps; a binary search is seven dependent loads)
  __device__ __forceinline__ int group_expert(const int* groups, int v) const {
    int n = 0;
#pragma unroll 1
    for (int e = threadIdx.x & 31; e < a.E; e += 32) n += groups[e] <= v ? 1 : 0;
    return __reduce_add_sync(0xffffffffu, n) - 1;
  }

  // The span that unit u begins or lies in: its units share tokens, expert and
  // reduction chunk, and differ by their rows.
  __device__ __forceinline__ Span span(int pass, int u, int last) const {
    Span q;
    const bool up = pass <= kUpRouted;
    const int ng = up ? a.ng_up : a.ng_down;
    const int per = up ? nfb : nb;
    int v = u / per;
    const int blk = u - v * per;
    q.units = min(per - blk, last - u);
    q.c = 0;
    if (!up && a.nc > 1) {
      const int t = v;
      v = t / a.nc;
      q.c = t - v * a.nc;
    }
    const char* base;
    if (pass == kUpShared || pass == kDownShared) {
      const int sg = up ? sg_up : sg_down;
      q.e = sg == 1 ? v : v / sg;
      q.row0 = (v - q.e * sg) * ng;
      q.n = min(ng, a.T - q.row0);
      base = up ? a.w13_s : a.w2_s;
    } else {
      const int* groups = s.groups[up ? 0 : 1];
      q.e = group_expert(groups, v);
      q.row0 = s.seg_off[q.e] + (v - groups[q.e]) * ng;
      q.n = min(ng, s.seg_off[q.e + 1] - q.row0);
      base = up ? a.w13 : a.w2;
    }
    if (up) {
      q.row_bytes = static_cast<int64_t>(a.d) * kW;
      q.step = 8;
      q.col = blk * 8;
      q.cols = a.F;
      q.len = a.d * kW;
      q.hi = a.F * q.row_bytes;
      q.w = base + (static_cast<int64_t>(q.e) * 2 * a.F + q.col) * q.row_bytes;
    } else {
      q.row_bytes = static_cast<int64_t>(a.F) * kW;
      q.step = kFewRows;
      q.col = blk * kFewRows;
      q.cols = a.d;
      const int64_t k0 = static_cast<int64_t>(q.c) * a.chunk_bytes;
      q.len = static_cast<int>(min(static_cast<int64_t>(a.chunk_bytes), q.row_bytes - k0));
      q.hi = 8 * q.row_bytes;
      q.w = base + (static_cast<int64_t>(q.e) * a.d + q.col) * q.row_bytes + k0;
    }
    return q;
  }
};

// A place in the CTA's list of units: the units of a pass, then those of the next.
template <int WT>
struct Place {
  int pass, u, last;
  __device__ __forceinline__ Place(const Few<WT>& f, int first_pass) : pass(first_pass) { enter(f); }
  __device__ __forceinline__ void enter(const Few<WT>& f) {
    const PassRange r = f.range(pass);
    u = r.first;
    last = r.last;
  }
  // whether a unit is left in the pass or, entering it, in the routed pass after it
  __device__ __forceinline__ bool more(const Few<WT>& f) {
    if (u >= last && (pass == kUpShared || pass == kDownShared)) {
      ++pass;
      enter(f);
    }
    return u < last;
  }
};

// The copy side (kCopiers warps, each its own rows of every stage; every lane
// of a warp holds the same Cursor).  Warps of their own: issuing the 16 copies
// of a stage takes some 800 cycles, which the products waited for while the same
// warps did both (32 tokens, d = 4096, E = 128: 1583 -> 781 us with one copying
// warp, 774 -> 648 us with two).  Each team has its own ring of kFewStages /
// teams stages, so that a team never waits for a phase of a barrier more than
// one ahead (a parity wait could not tell it from the past one).  The teams'
// units of a span are copied together, a stage of each in turn: stage k of
// units i, i + 1, then stage k + 1 of both.
struct Cursor {
  int pass = 0, u = 0, end = 0;  // next unit of the pass, the pass's last
  int left = 0, off = 0;         // units left in the span, bytes of the current units' rows copied
  int team = 0;                  // team whose stage is next
  uint32_t issued0 = 0, issued1 = 0;  // stages filled so far, by team
  Span q;
};

// Fill stages through pass last_pass (whose units are known by now); before the
// routing (kUpShared) only the stages that are free, afterwards waiting for each.
template <int WT>
__device__ __forceinline__ void few_fill(const Few<WT>& f, Cursor& c, int last_pass, int copier, int lane) {
  constexpr int kTeams = Few<WT>::kTeams, kSlots = kFewStages / kTeams;
  for (;;) {
    if (c.left == 0) {
      while (c.u >= c.end) {
        if (c.pass >= last_pass) return;
        ++c.pass;
        const PassRange r = f.range(c.pass);
        c.u = r.first;
        c.end = r.last;
      }
      c.q = f.span(c.pass, c.u, c.end);
      c.left = c.q.units;
      c.u += c.left;
      c.off = 0;
      c.team = 0;
    }
    const uint32_t issued = c.team ? c.issued1 : c.issued0;
    if (last_pass == kUpShared && issued >= kSlots) return;
    const int slot = c.team * kSlots + static_cast<int>(issued % kSlots);
    bool ok = true;
    if (issued >= kSlots) ok = mbar_wait(&f.s.empty[slot], (issued / kSlots - 1) & 1u, &f.s.abort_flag);
    if (!__all_sync(0xffffffffu, ok)) return;
    const int bytes = min(Few<WT>::kChunk, c.q.len - c.off);
    const int col = c.q.col + c.team * c.q.step;
    const int rows = c.q.step == 8 ? kFewRows : min(kFewRows, c.q.cols - col);
    uint64_t* bar = &f.s.full[slot];
    constexpr int kMine = kFewRows / Few<WT>::kCopiers;
    const int row = copier * kMine + lane;
    if (lane == 0) mbar_arrive_expect_tx(bar, static_cast<uint32_t>(max(0, min(kMine, rows - row)) * bytes));
    __syncwarp();
    if (lane < kMine && row < rows) {
      const char* src = c.q.w + (c.team * c.q.step + (row & 7)) * c.q.row_bytes + (row >> 3) * c.q.hi + c.off;
      bulk_load(f.ring + slot * Few<WT>::kStageBytes + row * Few<WT>::kPitch, src, static_cast<uint32_t>(bytes), bar);
    }
    if (c.team)
      ++c.issued1;
    else
      ++c.issued0;
    const int now = min(kTeams, c.left);  // units copied together
    if (++c.team >= now) {
      c.team = 0;
      c.off += bytes;
      if (c.off >= c.q.len) {
        c.left -= now;
        c.off = 0;
        c.q.col += now * c.q.step;
        c.q.w += now * c.q.step * c.q.row_bytes;
      }
    }
  }
}

// One stage's products (cb bytes of each row): acc += weights x tokens.
template <int WT>
struct FewMath;

// warp: the warp's place in its team.
template <int WT>
struct FewMathMma {
  using Acc = typename Few<WT>::Acc;
  static constexpr int kWarps = Few<WT>::kTeamWarps, kChunk = FewTile<WT>::kChunk, kPitch = FewTile<WT>::kPitch;
  static constexpr int kParts = Few<WT>::kParts;
  // [token tile][chain]: two chains of dependent products instead of one twice
  // as long
  Acc acc[2][2][4];
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[j >> 1][j & 1][i] = 0;
  }
  // w: the stage; t: the token buffer at the stage's first byte of the rows; low:
  // distance to the rows that are added to them, or 0
  __device__ __forceinline__ void stage(const uint8_t* w, const uint8_t* t, int t_pitch, int low, int cb, int n_tok,
                                        int rows, int warp, int lane) {
    // ldmatrix lane addresses: weights as four 8 x 16-byte blocks (rows 0-7 and
    // 8-15, bytes 0-15 and 16-31); tokens as 8 rows x 64 bytes
    const uint32_t wa = smem_addr(w) + (lane & 15) * kPitch + (lane >> 4) * 16;
    // (rows past the group's last repeat it: their sums are not read)
    const uint32_t ta = smem_addr(t) + min(lane & 7, n_tok - 1) * t_pitch + (lane >> 3) * 16;
    const uint32_t tb = smem_addr(t) + min(8 + (lane & 7), n_tok - 1) * t_pitch + (lane >> 3) * 16;
    if (cb == kChunk && rows == kFewRows) {
#pragma unroll
      for (int i = 0; i < kChunk / (64 * kWarps); ++i) {
        const int o = (i * kWarps + warp) * 64;
        uint32_t a0[4], a1[4];
        ldmatrix_x4(wa + o, a0);
        ldmatrix_x4(wa + o + 32, a1);
        tokens(ta + o, tb + o, low, n_tok, a0, a1);
      }
      return;
    }
    for (int o = warp * 64; o < cb; o += kWarps * 64) {
      uint32_t a0[4], a1[4];
      ldmatrix_x4(wa + o, a0);
      ldmatrix_x4(wa + o + 32, a1);
      if (o + 64 > cb) {  // the row ends inside: what lies behind it may be anything
        if (o + 16 >= cb) a0[2] = a0[3] = 0;
        if (o + 32 >= cb) a1[0] = a1[1] = 0;
        if (o + 48 >= cb) a1[2] = a1[3] = 0;
      }
      if (rows == 8) a0[1] = a0[3] = a1[1] = a1[3] = 0;
      tokens(ta + o, tb + o, low, n_tok, a0, a1);
    }
  }
  // 64 bytes of the tokens' rows with the weights a0 (bytes 0-31), a1 (32-63)
  __device__ __forceinline__ void tokens(uint32_t ta, uint32_t tb, int low, int n_tok, const uint32_t (&a0)[4],
                                         const uint32_t (&a1)[4]) {
    uint32_t b[4];
    ldmatrix_x4(ta, b);
    mma_16x8(acc[0][0], a0, b[0], b[1]);
    mma_16x8(acc[0][1], a1, b[2], b[3]);
    if (kParts > 1 && low) {
      ldmatrix_x4(ta + low, b);
      mma_16x8(acc[0][0], a0, b[0], b[1]);
      mma_16x8(acc[0][1], a1, b[2], b[3]);
    }
    if (n_tok > 8) {
      ldmatrix_x4(tb, b);
      mma_16x8(acc[1][0], a0, b[0], b[1]);
      mma_16x8(acc[1][1], a1, b[2], b[3]);
      if (kParts > 1 && low) {
        ldmatrix_x4(tb + low, b);
        mma_16x8(acc[1][0], a0, b[0], b[1]);
        mma_16x8(acc[1][1], a1, b[2], b[3]);
      }
    }
  }
  // this warp's sums to red[warp][tile][row][token]
  __device__ __forceinline__ void put(void* red, int n_tok, int warp, int lane) {
    Acc* r = static_cast<Acc*>(red) + warp * 256 + (lane >> 2) * 8 + (lane & 3) * 2;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      if (j * 8 >= n_tok) break;
      r[j * 128] = acc[j][0][0] + acc[j][1][0];
      r[j * 128 + 1] = acc[j][0][1] + acc[j][1][1];
      r[j * 128 + 64] = acc[j][0][2] + acc[j][1][2];
      r[j * 128 + 65] = acc[j][0][3] + acc[j][1][3];
    }
  }
  __device__ __forceinline__ static Acc get(const void* red, int row, int tok) {
    const Acc* r = static_cast<const Acc*>(red) + (tok >> 3) * 128 + row * 8 + (tok & 7);
    Acc v = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) v += r[w * 256];
    return v;
  }
};

template <>
struct FewMath<kFewBF16> : FewMathMma<kFewBF16> {};
template <>
struct FewMath<kFewBF16Many> : FewMathMma<kFewBF16Many> {};
template <>
struct FewMath<kFewI8> : FewMathMma<kFewI8> {};

// FP32: warp w takes rows (w >> 2) * 8 .. + 7 and the 512-byte slice w & 3 of a
// stage, a lane 16 bytes of it.
template <>
struct FewMath<kFewF32> {
  using Acc = float;
  float acc[8][8];
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int r = 0; r < 8; ++r)
#pragma unroll
      for (int j = 0; j < 8; ++j) acc[r][j] = 0.f;
  }
  __device__ __forceinline__ void stage(const uint8_t* w, const uint8_t* t, int t_pitch, int, int cb, int n_tok, int rows,
                                        int warp, int lane) {
    const int o = (warp & 3) * 512 + lane * 16;
    if (o >= cb || (warp >> 2) * 8 >= rows) return;
    constexpr int kPitch = FewTile<kFewF32>::kPitch;
    const uint8_t* wr = w + (warp >> 2) * 8 * kPitch + o;
    float4 wv[8];
#pragma unroll
    for (int r = 0; r < 8; ++r) wv[r] = *reinterpret_cast<const float4*>(wr + r * kPitch);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if (j < n_tok) {
        const float4 tv = *reinterpret_cast<const float4*>(t + j * t_pitch + o);
#pragma unroll
        for (int r = 0; r < 8; ++r) {
          acc[r][j] = fmaf(wv[r].x, tv.x, acc[r][j]);
          acc[r][j] = fmaf(wv[r].y, tv.y, acc[r][j]);
          acc[r][j] = fmaf(wv[r].z, tv.z, acc[r][j]);
          acc[r][j] = fmaf(wv[r].w, tv.w, acc[r][j]);
        }
      }
    }
  }
  // sum over the lanes by halving: lane l ends with entries 2l and 2l + 1 of [8 rows][8 tokens]
  __device__ __forceinline__ void put(void* red, int, int warp, int lane) {
    float v[64];
#pragma unroll
    for (int i = 0; i < 64; ++i) v[i] = acc[i >> 3][i & 7];
#pragma unroll
    for (int o = 16, m = 32; o > 0; o >>= 1, m >>= 1) {
#pragma unroll
      for (int i = 0; i < 32; ++i) {
        if (i < m) {
          const float send = (lane & o) ? v[i] : v[i + m];
          const float keep = (lane & o) ? v[i + m] : v[i];
          v[i] = keep + __shfl_xor_sync(0xffffffffu, send, o);
        }
      }
    }
    *reinterpret_cast<float2*>(static_cast<float*>(red) + warp * 64 + 2 * lane) = make_float2(v[0], v[1]);
  }
  __device__ __forceinline__ static float get(const void* red, int row, int tok) {
    const float* r = static_cast<const float*>(red) + (row >> 3) * 4 * 64 + (row & 7) * 8 + tok;
    return (r[0] + r[64]) + (r[128] + r[192]);
  }
};

// ---------------------------------------------------------------- token rows
// What the token buffer holds: the same rows need no second load (the shared
// experts: every group; one token: every expert's up product).
__device__ __forceinline__ int few_token_key(const FewArgs& a, int pass, const Span& q) {
  if (pass == kUpRouted && a.T == 1) return 1 << 16;
  return pass == kUpShared ? q.n << 16 | q.row0 : -1;
}

// distance of the rows in the token buffer: whole 64-byte slices, and an odd
// number of 16-byte pieces against bank conflicts
__device__ __forceinline__ int few_token_pitch(int len) { return ((len + 63) & ~63) + 16; }

// Rows of the span's group into the token buffer, zero behind the row's end up
// to the next multiple of 64 bytes.  up: rows of x (8-bit weights: its integers
// from step 1); down: a chunk of hidden rows (8-bit weights: FP32, rounded to
// integers here; every CTA has contributed to the row's largest magnitude).
// tok, row_scale: the span's first row and scale.  Rows that need no rounding
// are copied asynchronously: the caller waits.
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, int bytes) {  // the rest of 16: zero
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_async_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }

template <int WT>
__device__ __forceinline__ void few_load_tokens(const Few<WT>& f, int pass, const Span& q, uint8_t* tok,
                                                float* row_scale, int t_pitch, int tid) {
  const FewArgs& a = f.a;
  const bool up = pass <= kUpRouted;
  const bool routed = pass == kUpRouted || pass == kDownRouted;
  const int vecs = q.len / 16, all = ((q.len + 63) & ~63) / 16;
  const int n_rows = up ? q.n : q.n * Few<WT>::kParts;  // hidden rows: the high parts, then the low ones
  // 256 / (rows rounded up to a power of two) threads per row
  const int sh = __clz(n_rows - 1) - 24;
  const int per = 1 << sh, r = tid >> sh, v0 = tid & (per - 1);
  if (WT != kFewI8 || up) {
    if (r < n_rows) {
      const char* src;
      if (up) {
        src = static_cast<const char*>(WT == kFewI8 ? static_cast<const void*>(a.x_q) : a.x) +
              static_cast<int64_t>(routed ? f.s.perm[q.row0 + r] / a.K : q.row0 + r) * q.len;
      } else {
        const bool low = r >= q.n;
        int64_t row = q.row0 + (low ? r - q.n : r);
        if (!routed) row = row * a.Ns + q.e;
        if (low) row += f.low_rows(routed);
        src = static_cast<const char*>(routed ? a.h : a.h_s) + row * a.F * Few<WT>::kW +
              static_cast<int64_t>(q.c) * a.chunk_bytes;
      }
      const uint32_t dst = smem_addr(tok + r * t_pitch);
      for (int v = v0; v < all; v += per) {
        const bool in = v < vecs;
        cp_async16(dst + v * 16, src + (in ? v * 16 : 0), in ? 16 : 0);
      }
    }
    if (WT == kFewI8 && tid < q.n)
      row_scale[tid] = __ldcg(a.x_scale + (routed ? f.s.perm[q.row0 + tid] / a.K : q.row0 + tid));
  } else {
    if (r >= q.n) return;
    const int64_t row = q.row0 + r;
    const unsigned m = __ldcg(a.amax + (routed ? row : static_cast<int64_t>(a.T) * a.K + row));
    for (int v = v0; v < all; v += per) {
      const float4* src = reinterpret_cast<const float4*>(
          (routed ? static_cast<const float*>(a.h) + row * a.F
                  : static_cast<const float*>(a.h_s) + (row * a.Ns + q.e) * a.F) +
          static_cast<int64_t>(q.c) * a.chunk_bytes) + v * 4;
      uint32_t w[4] = {0, 0, 0, 0};
      float4 z[4];
      if (v < vecs) {
#pragma unroll
        for (int j = 0; j < 4; ++j) z[j] = __ldcg(src + j);
      }
      const float scale = quant_scale(m), inv = 1.0f / scale;
      if (v < vecs) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float e[4] = {z[j].x, z[j].y, z[j].z, z[j].w};
          w[j] = quant_pack4(e, scale, inv);
        }
      }
      *reinterpret_cast<uint4*>(tok + r * t_pitch + v * 16) = make_uint4(w[0], w[1], w[2], w[3]);
      if (v == 0) row_scale[r] = scale;
    }
  }
}

// 8-bit weights: the integers and the scale of token t (one CTA's workers).
__device__ __forceinline__ void few_quantize_token(const FewArgs& a, int t, unsigned* s_max, int tid) {
  const uint4* src = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.x) +
                                                    static_cast<int64_t>(t) * a.d);
  const int vecs = a.d / 8;
  unsigned m = 0;
#pragma unroll 4
  for (int v = tid; v < vecs; v += kFewWorkers) {
    const uint4 w = src[v];
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) m = max(m, max((u[i] << 16) & 0x7FFF0000u, u[i] & 0x7FFF0000u));
  }
  m = __reduce_max_sync(0xffffffffu, m);
  if ((tid & 31) == 0) s_max[tid >> 5] = m;
  named_bar_sync(1, kFewWorkers);
#pragma unroll
  for (int i = 0; i < kFewWorkers / 32; ++i) m = max(m, s_max[i]);
  const float scale = quant_scale(m), inv = 1.0f / scale;
  uint2* dst = reinterpret_cast<uint2*>(a.x_q + static_cast<int64_t>(t) * a.d);
#pragma unroll 4
  for (int v = tid; v < vecs; v += kFewWorkers) {
    const uint4 w = src[v];
    const float lo[4] = {bf16_lo(w.x), bf16_hi(w.x), bf16_lo(w.y), bf16_hi(w.y)};
    const float hi[4] = {bf16_lo(w.z), bf16_hi(w.z), bf16_lo(w.w), bf16_hi(w.w)};
    dst[v] = make_uint2(quant_pack4(lo, scale, inv), quant_pack4(hi, scale, inv));
  }
  if (tid == 0) a.x_scale[t] = scale;
  named_bar_sync(1, kFewWorkers);
}

// ------------------------------------------------------------- unit outputs
// 8-bit weights: the scales of the unit's rows that thread tid of the team
// stores, at row offset `ahead` (up: a gate and an up row; down: one channel).
template <int WT>
__device__ __forceinline__ float2 few_scales(const Few<WT>& f, int pass, const Span& q, int ahead, int tid) {
  const FewArgs& a = f.a;
  float2 v = make_float2(0.f, 0.f);
  if constexpr (WT == kFewI8) {
    if (pass <= kUpRouted) {
      const int col = q.col + ahead + (tid & 7);
      if (col < q.cols) {
        const float* sc = (pass == kUpShared ? a.s13_s : a.s13) + static_cast<int64_t>(q.e) * 2 * a.F + col;
        v.x = __ldg(sc);
        v.y = __ldg(sc + a.F);
      }
    } else {
      const int col = q.col + ahead + (tid & 15);
      if (col < q.cols) v.x = __ldg(pass == kDownShared ? a.s2_s + col : a.s2 + static_cast<int64_t>(q.e) * a.d + col);
    }
  }
  return v;
}

// sc: few_scales of this unit
template <int WT>
__device__ __forceinline__ void few_store_unit(const Few<WT>& f, int pass, const Span& q, const void* red, float2 sc,
                                               const float* row_scale, int tid) {
  using M = FewMath<WT>;
  const FewArgs& a = f.a;
  if (pass <= kUpRouted) {  // 8 features x n tokens: lane groups of 8 share a token
    const int ft = tid & 7, tok = tid >> 3;
    const bool live = tok < q.n;
    float h = 0.f;
    if (live) {
      if constexpr (WT == kFewI8) {
        const float sx = row_scale[tok];
        const float g = __int2float_rn(M::get(red, ft, tok)) * (sx * sc.x);
        const float u = __int2float_rn(M::get(red, ft + 8, tok)) * (sx * sc.y);
        h = silu(g) * u;
      } else {
        h = silu(M::get(red, ft, tok)) * M::get(red, ft + 8, tok);
      }
      const int64_t row = q.row0 + tok;
      const int64_t at = pass == kUpShared ? (row * a.Ns + q.e) * a.F + q.col + ft : row * a.F + q.col + ft;
      void* hp = pass == kUpShared ? a.h_s : a.h;
      if constexpr (Few<WT>::kParts == 2) {
        // h = high + low, off by at most 2^-16 of it: one BF16, the tensor cores'
        // operand, would put as much rounding into y as y's own (32 tokens,
        // d = 4096, E = 128 638 -> 654 us; one token, d = 2048 43.5 -> 45.4 us).  Infinities and NaN stay in the high part.
        const __nv_bfloat16 high = __float2bfloat16(h);
        const float rest = h - __bfloat162float(high);
        static_cast<__nv_bfloat16*>(hp)[at] = high;
        static_cast<__nv_bfloat16*>(hp)[at + f.low_rows(pass == kUpRouted) * a.F] =
            __float2bfloat16(isfinite(rest) ? rest : 0.f);
      } else {
        static_cast<float*>(hp)[at] = h;
      }
    }
    if constexpr (WT == kFewI8) {
      unsigned m = abs_bits(h);
#pragma unroll
      for (int o = 4; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o, 8));
      if (live && ft == 0)
        atomicMax(a.amax + (pass == kUpShared ? static_cast<int64_t>(a.T) * a.K : 0) + q.row0 + tok, m);
    }
  } else {  // 16 output channels x n tokens
    const int n = tid & 15;
    if (q.col + n >= q.cols) return;
    for (int tok = tid >> 4; tok < q.n; tok += Few<WT>::kTeamWarps * 2) {
      float v;
      if constexpr (WT == kFewI8)
        v = __int2float_rn(M::get(red, n, tok)) * (row_scale[tok] * sc.x);
      else
        v = M::get(red, n, tok);
      const int64_t row = q.row0 + tok;
      if (pass == kDownShared)
        a.part_s[((static_cast<int64_t>(q.e) * a.nc + q.c) * a.T + row) * a.d + q.col + n] = v;
      else
        a.part[(static_cast<int64_t>(q.c) * a.T * a.K + row) * a.d + q.col + n] = v;
    }
  }
}

// All units of two passes, first_pass (shared experts) and the next (routed
// ones), that are this CTA's (the 256 worker threads).  Team t takes units t,
// t + teams, ... of a span; `used`: stages this team has consumed.
template <int WT>
__device__ __forceinline__ void few_passes(const Few<WT>& f, int first_pass, uint32_t& used, uint8_t* red_base,
                                           uint32_t& n_units, int& held, int tid) {
  constexpr int kTeams = Few<WT>::kTeams, kWarps = Few<WT>::kTeamWarps, kSlots = kFewStages / kTeams;
  constexpr int kChunk = Few<WT>::kChunk;
  const int lane = tid & 31, team = (tid >> 5) / kWarps, warp = (tid >> 5) % kWarps;
  FewMath<WT> math;
  red_base += team * (kFewRedBytes / kTeams);
  const int parts = first_pass == kDownShared ? Few<WT>::kParts : 1;  // rows of a token in its buffer
  Place<WT> here(f, first_pass);
  int loaded = 0;           // spans, from this one on, whose rows are in the token buffer,
  int at = 0, row = 0;      // the next one's at byte `at`, their scales at `row`
  while (here.more(f)) {
    Span q = f.span(here.pass, here.u, here.last);
    const int pass = here.pass, t_pitch = few_token_pitch(q.len);
    here.u += q.units;
    if (loaded == 0) {
      at = row = 0;
      loaded = 1;
      const int key = few_token_key(f.a, pass, q);
      if (key < 0 || key != held) {
        // the last unit's reads of the token buffer (and of the row scales) are
        // over only once its outputs are stored
        named_bar_sync(1, kFewWorkers);
        // with as many of the next spans' rows as fit: a load costs 1.5 us of
        // latency and barriers
        Place<WT> p = here;
        Span n = q;
        int bytes = 0, rows = 0;
        for (;;) {
          const int pitch = few_token_pitch(n.len) * parts;
          few_load_tokens(f, p.pass, n, f.tok + bytes, f.s.row_scale + rows, few_token_pitch(n.len), tid);
          bytes += n.n * pitch;
          rows += n.n;
          if (key >= 0 || !p.more(f)) break;
          n = f.span(p.pass, p.u, p.last);
          if (rows + n.n > 16 || bytes + n.n * few_token_pitch(n.len) * parts > Few<WT>::kTokBytes) break;
          p.u += n.units;
          ++loaded;
        }
        cp_async_wait_all();
        named_bar_sync(1, kFewWorkers);
        held = key;
      }
    }
    --loaded;
    const uint8_t* tok = f.tok + at;
    const float* row_scale = f.s.row_scale + row;
    at += q.n * t_pitch * parts;
    const int low = parts > 1 ? q.n * t_pitch : 0;
    row += q.n;
    q.col += team * q.step;
    // 8-bit weights: the scales are fetched one unit ahead (fetched when needed
    // they cost the team a memory latency per unit: 210 -> 200 us for 7 tokens
    // of d = 4096, E = 128, F = 1536)
    const int team_tid = tid - team * kWarps * 32;
    float2 sc_next = few_scales(f, pass, q, 0, team_tid);
    for (int i = team; i < q.units; i += kTeams) {
      const float2 sc = sc_next;
      if (i + kTeams < q.units) sc_next = few_scales(f, pass, q, kTeams * q.step, team_tid);
      math.clear();
      uint8_t* red = red_base + (n_units & 1u) * (kFewRedBytes / kTeams / 2);
      const int rows = min(kFewRows, q.step == 8 ? kFewRows : q.cols - q.col);
      for (int off = 0; off < q.len; off += kChunk, ++used) {
        const int slot = team * kSlots + static_cast<int>(used % kSlots);
        mbar_wait(&f.s.full[slot], (used / kSlots) & 1u, &f.s.abort_flag);
        __syncwarp();
        math.stage(f.ring + slot * Few<WT>::kStageBytes, tok + off, t_pitch, low, min(kChunk, q.len - off), q.n, rows,
                   warp, lane);
        __syncwarp();
        if (lane == 0) mbar_arrive(&f.s.empty[slot]);
      }
      math.put(red, q.n, warp, lane);
      named_bar_sync(2 + team, kWarps * 32);  // the unit's sums are complete
      few_store_unit(f, pass, q, red, sc, row_scale, team_tid);
      q.col += kTeams * q.step;
      ++n_units;  // the next unit's sums go to the other half: no barrier before they are written
    }
  }
}

// ------------------------------------------------------------------- routing
// Tiles of 4 experts x 4 tokens: the 8 warps split d, a lane takes 16 bytes of
// each row per step, products are summed in FP32 per lane, the lanes and warps
// in FP64.
template <typename T>
__device__ __forceinline__ void few_logits(const FewArgs& a, double* red, int tid) {
  constexpr int V = 16 / static_cast<int>(sizeof(T));
  const int warp = tid >> 5, lane = tid & 31;
  const int te = (a.E + 3) / 4, tt = (a.T + 3) / 4;
  for (int tile = blockIdx.x; tile < te * tt; tile += gridDim.x) {
    const int e0 = (tile % te) * 4, t0 = (tile / te) * 4;
    float acc[4][4];
#pragma unroll
    for (int i = 0; i < 16; ++i) acc[i >> 2][i & 3] = 0.f;
    for (int k = (warp * 32 + lane) * V; k < a.d; k += kFewWorkers * V) {
      float w[4][V], x[4][V];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        // rows past the end repeat the last one; their sums are not stored
        const uint4 qw = *reinterpret_cast<const uint4*>(static_cast<const T*>(a.w_gate) +
                                                         static_cast<int64_t>(min(e0 + i, a.E - 1)) * a.d + k);
        const uint4 qx = *reinterpret_cast<const uint4*>(static_cast<const T*>(a.x) +
                                                         static_cast<int64_t>(min(t0 + i, a.T - 1)) * a.d + k);
        if constexpr (sizeof(T) == 2) {
          unpack16(qw, w[i], static_cast<const __nv_bfloat16*>(nullptr));
          unpack16(qx, x[i], static_cast<const __nv_bfloat16*>(nullptr));
        } else {
          w[i][0] = __uint_as_float(qw.x); w[i][1] = __uint_as_float(qw.y);
          w[i][2] = __uint_as_float(qw.z); w[i][3] = __uint_as_float(qw.w);
          x[i][0] = __uint_as_float(qx.x); x[i][1] = __uint_as_float(qx.y);
          x[i][2] = __uint_as_float(qx.z); x[i][3] = __uint_as_float(qx.w);
        }
      }
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int v = 0; v < V; ++v) acc[i][j] = fmaf(w[i][v], x[j][v], acc[i][j]);
    }
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const double s = warp_sum(static_cast<double>(acc[i >> 2][i & 3]));
      if (lane == 0) red[warp * 16 + i] = s;
    }
    named_bar_sync(1, kFewWorkers);
    if (tid < 16) {
      const int e = e0 + (tid >> 2), t = t0 + (tid & 3);
      if (e < a.E && t < a.T) {
        double s = 0.0;
        for (int w = 0; w < 8; ++w) s += red[w * 16 + tid];
        a.logits[static_cast<int64_t>(t) * a.E + e] =
            static_cast<float>(s + (a.logit_offset ? static_cast<double>(a.logit_offset[e]) : 0.0));
      }
    }
    named_bar_sync(1, kFewWorkers);
  }
}

// Softmax and top-K of tokens first, first + step, ... (one warp), into idx / w
// [T K]; stats: also the sums of p and the squared logsumexp.
template <int EPL>
__device__ __forceinline__ void few_select(const FewArgs& a, FewShared& s, int32_t* idx, float* w, bool with_stats,
                                           int first, int step, int lane) {
  float bias[EPL];
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
    const int e = lane + 32 * i;
    bias[i] = (a.sel_bias && e < a.E) ? a.sel_bias[e] : 0.f;
  }
#pragma unroll 1
  for (int t = first; t < a.T; t += step) {
    float lg[EPL], p[EPL], zacc = 0.f;
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      const int e = lane + 32 * i;
      lg[i] = e < a.E ? __ldcg(a.logits + static_cast<int64_t>(t) * a.E + e) : -INFINITY;
      p[i] = 0.f;
    }
    select_token_group<EPL, 32>(lg, bias, a.sel_bias != nullptr, a.bias_on_logit, a.E, a.K, lane, p, zacc,
                                idx + t * a.K, w + t * a.K, s.counts);
    if (with_stats) {
      if (lane == 0) a.lse2[t] = zacc;
#pragma unroll
      for (int i = 0; i < EPL; ++i)
        if (lane + 32 * i < a.E && p[i] > 0.f)
          atomicAdd(a.psum + lane + 32 * i, __double2ull_rn(static_cast<double>(p[i]) * a.pscale));
    }
  }
}

__device__ __forceinline__ void few_select_any(const FewArgs& a, FewShared& s, int32_t* idx, float* w,
                                               bool with_stats, int first, int step, int lane) {
  if (a.E <= 32)
    few_select<1>(a, s, idx, w, with_stats, first, step, lane);
  else if (a.E <= 64)
    few_select<2>(a, s, idx, w, with_stats, first, step, lane);
  else if (a.E <= 128)
    few_select<4>(a, s, idx, w, with_stats, first, step, lane);
  else
    few_select<8>(a, s, idx, w, with_stats, first, step, lane);
}

// Capacity, slots and the experts' token groups from idx (the 256 workers).
// The token's rank within its expert is the number of earlier tokens in the
// expert's bit mask.  (Written with few instructions: the code runs once, and
// fetching it costs more than executing it.)
__device__ __forceinline__ void few_dispatch(const FewArgs& a, FewShared& s, const int32_t* idx, const float* w,
                                             bool write, int tid) {
  static_assert(kMaxExperts == kFewWorkers, "one worker thread per expert");
  const int TK = a.T * a.K, lane = tid & 31;
#pragma unroll 1
  for (int i = tid; i < TK; i += kFewWorkers) {
    const unsigned e = static_cast<unsigned>(idx[i]), t = static_cast<unsigned>(i) / a.K;
    // 32-bit halves: a native shared-memory atomic
    if (e < static_cast<unsigned>(a.E)) atomicOr(reinterpret_cast<unsigned*>(&s.mask[e]) + (t >> 5), 1u << (t & 31));
  }
  named_bar_sync(1, kFewWorkers);
  // thread e: the expert's rows and token groups; one scan over the experts of
  // the three counts, 20 bits each (at most 2048 rows in all)
  const int n = __popcll(s.mask[tid]);
  int k = 0;
  if (tid < a.E) {
    long long cap = a.cap;
    if (a.expert_cap) cap = a.expert_cap[tid];
    k = (cap < 0 || n < cap) ? n : static_cast<int>(cap);
    s.kept[tid] = k;
    s.counts[tid] = n;
  }
  const unsigned long long mine = static_cast<unsigned long long>(k) |
                                  static_cast<unsigned long long>((k + a.ng_up - 1) / a.ng_up) << 20 |
                                  static_cast<unsigned long long>((k + a.ng_down - 1) / a.ng_down) << 40;
  unsigned long long incl = mine;
#pragma unroll 1
  for (int o = 1; o < 32; o <<= 1) {
    const unsigned long long v = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += v;
  }
  if (lane == 31) s.scan[tid >> 5] = incl;
  named_bar_sync(1, kFewWorkers);
#pragma unroll 1
  for (int i = 0; i < (tid >> 5); ++i) incl += s.scan[i];
  const unsigned long long excl = incl - mine;
  const int off = static_cast<int>(excl & 0xFFFFFu);
  s.seg_off[tid] = off;
  s.groups[0][tid] = static_cast<int>((excl >> 20) & 0xFFFFFu);
  s.groups[1][tid] = static_cast<int>(excl >> 40);
  // (an expert past the last has no rows, so entry E is the total)
  if (tid == kMaxExperts - 1) {
    s.seg_off[kMaxExperts] = static_cast<int>(incl & 0xFFFFFu);
    s.groups[0][kMaxExperts] = static_cast<int>((incl >> 20) & 0xFFFFFu);
    s.groups[1][kMaxExperts] = static_cast<int>(incl >> 40);
  }
  if (write && tid < a.E) {
    a.counts[tid] = n;
    a.kept[tid] = k;
    a.seg_off[tid] = off;
    if (tid == a.E - 1) a.seg_off[a.E] = off + k;
  }
  named_bar_sync(1, kFewWorkers);
#pragma unroll 1
  for (int i = tid; i < TK; i += kFewWorkers) {
    const unsigned e = static_cast<unsigned>(idx[i]), t = static_cast<unsigned>(i) / a.K;
    int slot = -1;
    if (e < static_cast<unsigned>(a.E)) {
      const int rank = __popcll(s.mask[e] & ((1ull << t) - 1ull));
      if (rank < s.kept[e]) slot = s.seg_off[e] + rank;
    }
    if (slot >= 0) s.perm[slot] = static_cast<uint16_t>(i);
    if (write) {
      a.slot_of[i] = slot;
      if (slot >= 0) a.perm[slot] = i;
      if (w) {
        a.topk_idx[i] = static_cast<int>(e);
        a.topk_w[i] = w[i];
      }
    }
  }
}

// y_t = sum over the shared experts' chunks + sum_k w_k (sum of Expert_k's
// chunks), k ascending; the loads of four addends at a time are in flight.
// slot, w: the tokens' slots and gates in shared memory.
template <typename T>
__device__ __forceinline__ void few_combine(const FewArgs& a, const int32_t* slot, const float* w, int tid) {
  // four: the code runs once and is fetched from memory (the weights' stream
  // evicts it between calls), so more unrolling costs more than it overlaps
  // (eight 4.0 us, twelve 6.4 us for one token, d = 2048, 12 addends)
  constexpr int kFly = 4;
  const int vecs = a.d / 4;
  const int total = a.T * vecs;
#pragma unroll 1
  for (int i = blockIdx.x * kFewWorkers + tid; i < total; i += gridDim.x * kFewWorkers) {
    const int t = i / vecs, c = (i - t * vecs) * 4;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f), e = acc;
    // addends: the shared experts' chunks, then each choice's
    const int ns = a.Ns * a.nc, nr = ns + a.K * a.nc;
    int n = 0, k = 0;
#pragma unroll 1
    for (int m0 = 0; m0 < nr; m0 += kFly) {
      float4 v[kFly];
      int of[kFly];  // choice the addend ends, or -1
#pragma unroll
      for (int j = 0; j < kFly; ++j) {
        const int m = m0 + j;
        v[j] = make_float4(0.f, 0.f, 0.f, 0.f);
        of[j] = -1;
        if (m < ns) {
          v[j] = __ldcg(reinterpret_cast<const float4*>(a.part_s + (static_cast<int64_t>(m) * a.T + t) * a.d + c));
        } else if (m < nr) {
          const int sl = slot[t * a.K + k];
          if (sl >= 0)
            v[j] = __ldcg(reinterpret_cast<const float4*>(a.part + (static_cast<int64_t>(n) * a.T * a.K + sl) * a.d + c));
          if (++n == a.nc) {
            of[j] = sl >= 0 ? k : -1;
            n = 0;
            ++k;
          }
        }
      }
#pragma unroll
      for (int j = 0; j < kFly; ++j) {
        if (m0 + j < ns) {
          acc.x += v[j].x; acc.y += v[j].y; acc.z += v[j].z; acc.w += v[j].w;
        } else {
          e.x += v[j].x; e.y += v[j].y; e.z += v[j].z; e.w += v[j].w;
          if (of[j] >= 0) {
            const float g = w[t * a.K + of[j]];
            acc.x = fmaf(g, e.x, acc.x); acc.y = fmaf(g, e.y, acc.y);
            acc.z = fmaf(g, e.z, acc.z); acc.w = fmaf(g, e.w, acc.w);
            e = make_float4(0.f, 0.f, 0.f, 0.f);
          }
        }
      }
    }
    T* yp = static_cast<T*>(a.y) + static_cast<int64_t>(t) * a.d + c;
    if constexpr (sizeof(T) == 2)
      *reinterpret_cast<uint2*>(yp) = make_uint2(pack_bf16x2(acc.x, acc.y), pack_bf16x2(acc.z, acc.w));
    else
      *reinterpret_cast<float4*>(yp) = acc;
  }
}

template <int WT>
__global__ void __launch_bounds__(FewTile<WT>::kThreads, 1) few_layer_kernel(const __grid_constant__ FewArgs a) {
  using X = typename std::conditional<WT == kFewF32, float, __nv_bfloat16>::type;
  extern __shared__ uint8_t few_smem[];
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(few_smem) + 127) & ~uintptr_t(127));
  uint8_t* ring = base;
  constexpr int kThreads = FewTile<WT>::kThreads, kCopiers = FewTile<WT>::kCopiers;
  uint8_t* tok = ring + kFewStages * FewTile<WT>::kStageBytes;
  uint8_t* red = ring + kFewBufBytes;
  FewShared& s = *reinterpret_cast<FewShared*>(red + kFewRedBytes);
  cg::grid_group grid = cg::this_grid();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int copier = warp - kFewWorkers / 32;  // 0 .. kCopiers - 1: a copying warp
  const bool worker = copier < 0, copies = copier >= 0 && copier < kCopiers;

  if (tid == 0) {
    for (int i = 0; i < kFewStages; ++i) {
      mbar_init(&s.full[i], kCopiers);
      mbar_init(&s.empty[i], Few<WT>::kTeamWarps);
    }
    mbar_init(&s.never, 1);
    s.abort_flag = 0;
    fence_barrier_init();
  }
  for (int i = tid; i < kMaxExperts; i += kThreads) {
    s.mask[i] = 0;
    if (blockIdx.x == 0 && i < a.E) a.psum[i] = 0;
  }
  if (blockIdx.x == 0 && tid < 3) a.arrivals[tid] = 0;
  if (blockIdx.x == 0 && tid == 0) *a.status = 0;
  if (WT == kFewI8) {
    for (int i = blockIdx.x * kThreads + tid; i < a.T * a.K + a.T; i += gridDim.x * kThreads) a.amax[i] = 0;
  }
  __syncthreads();

  const Few<WT> f(a, s, ring, tok);
  Cursor cur;
  uint32_t used = 0, n_units = 0;
  int held = -1;
  if (copies) {  // the shared experts' weights do not wait for the routing
    const PassRange r = f.range(kUpShared);
    cur.u = r.first;
    cur.end = r.last;
    few_fill(f, cur, kUpShared, copier, lane);
  }
  if (worker) {
    if (!a.given) few_logits<X>(a, reinterpret_cast<double*>(red), tid);
    if constexpr (WT == kFewI8) {  // the last CTAs first: the first ones have the logits' tiles
      for (int t = gridDim.x - 1 - blockIdx.x; t < a.T; t += gridDim.x)
        few_quantize_token(a, t, reinterpret_cast<unsigned*>(red), tid);
    }
  }
  grid.sync();

  bool go = true;  // false: a wait was given up (workers; the same in all of them)
  // the tests' stalled run: CTA 0 comes late, the other CTAs wait a quarter of that
  const unsigned long long limit_ns = a.stall_ns ? a.stall_ns / 4 : kWaitLimitNs;
  if (a.stall_ns && blockIdx.x == 0 && tid == 0) test_stall(&s.never, &s.abort_flag, a.stall_ns);
  if (worker) {
    int32_t* idx = reinterpret_cast<int32_t*>(tok);
    const bool write = blockIdx.x == 0;
    float* w = reinterpret_cast<float*>(tok) + kFewMaxPairs;
    // (one call: the code of two would be fetched from memory twice as often)
    few_select_any(a, s, a.spread ? a.topk_idx : idx, a.spread ? a.topk_w : w, a.stats && (a.spread || write),
                   a.spread ? blockIdx.x + warp * gridDim.x : warp, (a.spread ? gridDim.x : 1) * (kFewWorkers / 32),
                   lane);
    if (a.spread) {
      // (given up: some entries may be missing; few_dispatch takes any values, and
      // the copying warps need the counts that it makes)
      go = few_grid_sync(a.arrivals, s, limit_ns, tid);
#pragma unroll 1
      for (int i = tid; i < a.T * a.K; i += kFewWorkers) idx[i] = __ldcg(a.topk_idx + i);
    }
    named_bar_sync(1, kFewWorkers);
    few_dispatch(a, s, idx, a.spread ? nullptr : w, write, tid);
  }
  __syncthreads();
  if (worker) {
    // one copy of the code for all passes: what runs for the first time is
    // fetched from memory first (the weights' stream evicts it between calls)
#pragma unroll 1
    for (int pass = kUpShared; pass <= kDownShared; pass += kDownShared - kUpShared) {
      if (pass == kDownShared) go = few_grid_sync(a.arrivals + 1, s, limit_ns, tid);
      if (go) few_passes(f, pass, used, red, n_units, held, tid);
    }
    // the gates and slots of the combine, while the other CTAs finish
    named_bar_sync(1, kFewWorkers);
    int32_t* slot = reinterpret_cast<int32_t*>(tok);
    float* gate = reinterpret_cast<float*>(tok) + kFewMaxPairs;
#pragma unroll 1
    for (int i = tid; i < a.T * a.K; i += kFewWorkers) {
      // (CTA 0 wrote them before the barrier behind the up pass; no value, not
      // even one that it had no time to write, is used as a row that is not there)
      const int sl = __ldcg(a.slot_of + i);
      slot[i] = static_cast<unsigned>(sl) < static_cast<unsigned>(s.seg_off[a.E]) ? sl : -1;
      gate[i] = __ldcg(a.topk_w + i);
    }
    go = few_grid_sync(a.arrivals + 2, s, limit_ns, tid);
    if (go) few_combine<X>(a, slot, gate, tid);
  } else if (copies) {
    few_fill(f, cur, kDownRouted, copier, lane);
  } else if (blockIdx.x == 0 && a.stats) {
    // the statistics, beside the other warps' work
    for (int e = lane; e < a.E; e += 32)
      s.fp[e] = balance_stats_expert(s.counts[e], __ldcg(a.psum + e), a.T, a.E, a.K, e, a.stats);
    __syncwarp();
    if (lane == 0) {
      balance_loss(s.fp, a.E, a.alpha, a.stats);
      if (a.extended) {
        double z = 0.0;
        for (int t = 0; t < a.T; ++t) z += __ldcg(a.lse2 + t);
        utilisation_stats(s.counts, s.kept, a.E, a.T, z, a.stats);
      }
    }
  }
  __syncthreads();
  if (*static_cast<volatile int*>(&s.abort_flag)) {
    if (tid == 0) raise_status(a.status, kDevWaitTimeout);
    if (copies && lane == 0) {
      // nobody may have waited for the last copies: let each land before the block ends
      constexpr uint32_t kSlots = kFewStages / Few<WT>::kTeams;
      int late = 0;
      for (int t = 0; t < Few<WT>::kTeams; ++t) {
        const uint32_t n = t ? cur.issued1 : cur.issued0;
        for (uint32_t i = n > kSlots ? n - kSlots : 0; i < n; ++i)
          mbar_wait(&s.full[t * kSlots + i % kSlots], (i / kSlots) & 1u, &late);
      }
    }
  }
}

// ----------------------------------------------------------------- host side
static int64_t few_pitch(int64_t bytes) { return ((bytes + 63) & ~int64_t(63)) + 16; }

static size_t few_weight_bytes(const Problem& p, bool i8) { return i8 ? 1 : p.esize(); }

bool few_supported(const Problem& p, bool i8) {
  if (p.T > kFewMaxTokens) return false;
  if (few_pitch(static_cast<int64_t>(p.d) * few_weight_bytes(p, i8)) > FewTile<kFewI8>::kTokBytes) return false;
  // units are counted in 32 bits: at most one group per row
  const int64_t rows = p.T * p.K > p.T * p.Ns ? p.T * p.K : p.T * p.Ns;
  const int64_t lim = int64_t(1) << 31;
  const int64_t chunks = static_cast<int64_t>(p.F) * 4 / 2048 + 1;
  return rows * (p.F / 8) < lim && rows * chunks < lim && rows * chunks * (p.d / 8) < lim;
}

// Rows per token group and reduction chunks: as many rows as the token buffer
// and the two 8-token tiles hold.  A chunk of the down product's reduction is
// as long as leaves room for min(T, 8) rows, at most 8 KB.
static void few_tiling(const Problem& p, bool i8, int tok_bytes, FewArgs* a) {
  const int64_t ws = static_cast<int64_t>(few_weight_bytes(p, i8));
  const int64_t most = p.dtype == kF32 && !i8 ? 8 : 16;
  auto rows = [&](int64_t bytes, int parts) {
    const int64_t n = tok_bytes / (few_pitch(bytes) * parts);
    return static_cast<int>(n < most ? n : most);
  };
  const int parts = p.dtype == kBF16 && !i8 ? 2 : 1;  // of a hidden value
  a->ng_up = rows(p.d * ws, 1);
  const int64_t fb = p.F * ws;
  const int64_t want = (p.T < 8 ? p.T : 8) * parts;
  int64_t longest = (FewTile<kFewBF16>::kTokBytes / want - 80) / 2048 * 2048;
  // 8 KB give every CTA many units: with one chunk of 28 KB (F = 14336, one
  // token) a CTA had 3 or 4 units and the down product ended 15% late
  if (longest > 8192) longest = 8192;
  a->nc = static_cast<int>((fb + longest - 1) / longest);
  const int64_t even = (fb + a->nc - 1) / a->nc;
  const int64_t chunk = (even + 63) / 64 * 64;  // chunks of equal length: units of equal cost
  a->nc = static_cast<int>((fb + chunk - 1) / chunk);
  a->chunk_bytes = static_cast<int>(chunk);
  a->ng_down = rows(fb < chunk ? fb : chunk, parts);
}

// Reads of the experts' weights, about: an expert whose rows do not fit one
// token group is read once per group.
static double few_reads(const Problem& p, const FewArgs& a) {
  const double r = static_cast<double>(p.T * p.K) / p.E;  // rows of an expert on average
  auto groups = [](double rows, int ng) { return rows <= 0.5 * ng ? 1.0 : rows / ng + 0.5; };
  const double live = p.T * p.K < p.E ? static_cast<double>(p.T * p.K) : static_cast<double>(p.E);
  const double sh = p.Ns;
  auto whole = [&](int ng) { return static_cast<double>((p.T + ng - 1) / ng); };
  return 2.0 * (live * groups(r, a.ng_up) + sh * whole(a.ng_up)) + live * groups(r, a.ng_down) + sh * whole(a.ng_down);
}

FewLayout make_few_layout(const Problem& p) {
  FewLayout L{};
  size_t off = 0;
  auto take = [&](size_t bytes) {
    const size_t o = off;
    off = (off + (bytes ? bytes : 1) + 255) & ~size_t(255);
    return o;
  };
  const size_t T = static_cast<size_t>(p.T), TK = T * p.K;
  // 8-bit weights keep the hidden rows in FP32 and may need more chunks
  FewArgs a{}, b{};
  few_tiling(p, false, FewTile<kFewBF16>::kTokBytes, &a);
  few_tiling(p, true, FewTile<kFewI8>::kTokBytes, &b);
  const size_t nc = static_cast<size_t>(a.nc > b.nc ? a.nc : b.nc);
  L.status = take(256);
  L.logits = take(T * p.E * 4);
  L.topk_idx = take(TK * 4);
  L.topk_w = take(TK * 4);
  L.counts = take(static_cast<size_t>(p.E) * 4);
  L.kept = take(static_cast<size_t>(p.E) * 4);
  L.seg_off = take(static_cast<size_t>(p.E + 1) * 4);
  L.slot_of = take(TK * 4);
  L.perm = take(TK * 4);
  L.psum = take(static_cast<size_t>(p.E) * 8);
  L.lse2 = take(T * 4);
  L.x_q = take(T * p.d);
  L.x_scale = take(T * 4);
  L.amax = take((TK + T) * 4);
  L.h = take(TK * p.F * 4);
  L.h_s = take(T * p.Ns * p.F * 4);
  L.part = take(nc * TK * p.d * 4);
  L.part_s = take(nc * T * p.Ns * p.d * 4);
  L.total = off;
  return L;
}

template <int WT>
static cudaError_t run_few(const FewArgs& a, int64_t ctas, cudaStream_t st) {
  constexpr int smem = few_smem_bytes();
  static std::mutex mu;
  static uint64_t done = 0;
  int dev = 0;
  if (cudaError_t e = cudaGetDevice(&dev)) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  {
    std::lock_guard<std::mutex> lock(mu);
    if (!((done >> dev) & 1u)) {
      if (cudaError_t e = cudaFuncSetAttribute(few_layer_kernel<WT>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem))
        return e;
      done |= uint64_t(1) << dev;
    }
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(ctas));
  cfg.blockDim = dim3(FewTile<WT>::kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeCooperative;
  attr[0].val.cooperative = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, few_layer_kernel<WT>, a);
  if (e != cudaSuccess) cudaGetLastError();  // reported to the caller, not left for the next CUDA call
  return e;
}

cudaError_t launch_few_layer(const Problem& p, const FewCall& c, cudaStream_t st) {
  FewArgs a{};
  a.x = c.x;
  a.w_gate = c.w_gate;
  a.logit_offset = c.logit_offset;
  a.sel_bias = c.sel_bias;
  a.expert_cap = c.expert_cap;
  a.w13 = static_cast<const char*>(c.w13);
  a.w2 = static_cast<const char*>(c.w2);
  a.w13_s = static_cast<const char*>(c.w13_s);
  a.w2_s = static_cast<const char*>(c.w2_s);
  a.s13 = c.s13;
  a.s2 = c.s2;
  a.s13_s = c.s13_s;
  a.s2_s = c.s2_s;
  a.y = c.y;
  a.logits = c.logits;
  a.topk_idx = c.topk_idx;
  a.topk_w = c.topk_w;
  a.counts = c.counts;
  a.kept = c.kept;
  a.seg_off = c.seg_off;
  a.slot_of = c.slot_of;
  a.perm = c.perm;
  a.stats = c.stats;
  a.h = c.h;
  a.h_s = c.h_s;
  a.x_q = c.x_q;
  a.x_scale = c.x_scale;
  a.amax = c.amax;
  a.part = c.part;
  a.part_s = c.part_s;
  a.status = c.status;
  a.arrivals = c.status + 16;
  a.psum = c.psum;
  a.lse2 = c.lse2;
  a.spread = p.T > kFewWorkers / 32;
  a.T = static_cast<int>(p.T);
  a.d = p.d;
  a.E = p.E;
  a.K = p.K;
  a.Ns = p.Ns;
  a.F = p.F;
  a.cap = p.cap;
  a.given = c.given ? 1 : 0;
  a.bias_on_logit = (p.flags & 0x2u) ? 1 : 0;
  a.extended = (p.flags & 0x4u) ? 1 : 0;
  a.alpha = p.alpha;
  a.pscale = p_fixed_scale(p.T);
  a.stall_ns = test_stall_ns();
  few_tiling(p, c.i8, FewTile<kFewBF16>::kTokBytes, &a);
  // BF16 rows of more than 4 KB: 16 rows fit the token buffer only with half the
  // ring, whose stream is some 15% slower.  Taken when that saves 23% of the reads;
  // us without / with it, by the share of the reads that is left:
  //   0.58  d = 6144, E = 8,  F = 8192,  top-2,     64 tokens  1165 / 879
  //   0.60  d = 4096, E = 8,  F = 14336, top-2,     64 tokens   952 / 767
  //   0.67  the same,                               32 tokens   591 / 563
  //   0.75  d = 2816, E = 16, F = 5632,  top-2 + 1, 64 tokens   437 / 419
  //   0.79  d = 4096, E = 16, F = 4096,  top-2 + 2, 40 tokens   417 / 430
  //   0.80  d = 4096, E = 8,  F = 14336, top-2,     24 tokens   484 / 561
  //   0.98  d = 4096, E = 128, F = 1536, top-8 + 1, 64 tokens   825 / 945
  bool many = false;
  if (!c.i8 && p.dtype == kBF16) {
    FewArgs m = a;
    few_tiling(p, false, FewTile<kFewBF16Many>::kTokBytes, &m);
    if (few_reads(p, m) < 0.77 * few_reads(p, a)) {
      a = m;
      many = true;
    }
  }
  // one CTA per SM, or one per unit of the smaller problems
  const int64_t TK = p.T * p.K;
  int64_t units = (p.F / 8) * ((TK < p.E ? TK : p.E) + (TK + a.ng_up - 1) / a.ng_up + p.Ns * ((p.T + a.ng_up - 1) / a.ng_up));
  int64_t ctas = num_sms();
  if (units < ctas) ctas = units;
  if (ctas < 1) ctas = 1;
  if (c.i8) return run_few<kFewI8>(a, ctas, st);
  if (p.dtype == kF32) return run_few<kFewF32>(a, ctas, st);
  return many ? run_few<kFewBF16Many>(a, ctas, st) : run_few<kFewBF16>(a, ctas, st);
}

}  // namespace moe
