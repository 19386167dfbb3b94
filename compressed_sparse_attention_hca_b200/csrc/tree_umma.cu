// tree_umma.cu -- attention of a tree of drafted tokens on the 5th-generation
// tensor cores, for c = 512 and head counts that are a multiple of 64
// ("DeepSeek-V4 内部机制" 1.2 Step 2 shared-KV MQA, 1.3 HCA, 1.4 window branch
// and sink equation; yunpan.plus eq. 9).
//
// A node (drafted token) and 64 of its heads are a unit of work.  Its rows --
// entries, committed window tokens, drafted rows of its mask -- are taken 128
// at a time (a chunk).  As each row is both key and value, one tile in shared
// memory serves both products:
//   S^T[128 rows, 64 heads]  = K[128, 512] Q[64, 512]^T    (tile K-major)
//   O^T[512 dims, 64 heads] += V^T[512, 128] P^T[128, 64]  (tile MN-major)
// with O^T in 256 columns of TMEM.  A 128 x 64 x 16 product reads 6 KB of
// shared memory, 48 cycles at 128 bytes each (measured: 48.3) where the math
// takes 32, so a chunk's 64 products take 3,100; filling the tile takes 2,000
// (66 bytes a cycle from L2 with all SMs at it) behind a latency of 1,600.
// There is room for one tile, so a chunk is a chain.  96 or 128 heads would not
// fit TMEM next to O^T (4 x 128 columns) or shared memory.  Measured: 5,200
// cycles a chunk of BF16 rows, 7,000 of FP8MIX rows, whose decoding the softmax
// warps do too.  8 requests x 16 tokens over 1M tokens of HCA (131 GFLOP) take
// 185 us, with FP8MIX rows 280; the math alone at the bf16 rate would take 80,
// the products at their shared-memory rate ~100.  Small calls are bound by what
// surrounds the chunks: ~6,000 cycles of set-up, 2,500 to look up the first
// rows, 4,000 for the output, and the combine kernel's 3 us (one request of 3
// tokens: 14.6 us).  All of it waits for instructions more than for anything
// else: the roles' code overflows the first-level instruction cache, so loops
// are kept short.
//
// A chunk is a chain: S^T, softmax, O^T, and the four pairs of 64-dim atoms of
// the next chunk as those of this one are read.  One thread issues all
// products.  Eight warps take the softmax and then, idle until the next S^T,
// fill the tile; a warp looks up the rows' addresses up to three chunks ahead,
// and two load the queries and, of FP8MIX rows, decode the scales and the last
// pair.  (Chunks of 112 rows, which leave room for a fifth pair, were slower:
// 58 cycles a row against 48.)  The softmax is kept short: P is formed against
// the maximum of earlier chunks, and only a vote that finds a logit above it by
// more than 14 (log2) makes the warps find the new maximum, rescale what was
// summed, and form P again.  The sums of P stay in registers, a row per lane,
// until the end of the unit.
//
// P is rounded to the type of the rows, as an MMA's operands have one type: to
// bf16 for BF16 rows (2^-8 a weight, where the output's rounding is as much
// again: 0.0022 of the output in the root mean square, 0.0017 from the output
// alone), to fp16 for FP8MIX rows (2^-11).
//
// (TMA gathers of 4 x 128 bytes took 14,900 cycles a chunk, as every bulk
// instruction costs ~57 cycles whatever its size.)
//
// FP8MIX rows are decoded into an fp16 tile: value = code * scale has 24
// significant bits, which bf16 would cut to 8 (2^-8 of every key, value and
// weight; fp16: 2^-11), and the decoding is one conversion and one product per
// two values.  A power of two per row, 2^e, keeps the row in fp16's range, and
// is put back where it costs nothing: on the row's logits, and in the exponent
// of its weights.  P' = 2^(s + e - M) then carries it to O^T, M being the
// maximum of s + e.  The sums take 2^(s - M): 2^-e P', or of rows so small that
// P' may have been flushed to 0 where 2^(s - M) counts (e < -18: a row below
// 2^-3 or so, or of zeros) their logits once more (HCA at 1M with one row in 100
// of zeros: 280 us against 277).  e is at least -80, so that 2^30 rows of
// 2^(s - M) <= 2^(14 + 80) stay in fp32's range.  The query is scaled by a power
// of two per unit likewise.
//
// Work split: units are cut where the flattened list of all units' chunks is
// cut into equal parts, one per SM, so ragged contexts load the SMs evenly; a
// part writes the units that it holds whole and leaves partials of the others
// for the combine kernel: o / l in fp16 with a power of two per dim (2^-11;
// fp32 partials took twice the traffic, bf16 ones added as much error as the
// output's own rounding), and (m, l) in fp32.  Many units (8 per SM) are dealt
// out whole; a fixed split count cuts each unit by its own rows alone.
#include <cuda_fp16.h>

#include "csa_internal.cuh"
#include "mqa_plan.cuh"
#include "rope_dev.cuh"
#include "sm100.cuh"

namespace csa {

CSA_DEFINE_STATUS_READER(take_status_tree_umma)

namespace {

constexpr int kDim = 512;
constexpr int kHG = 64;      // heads per unit (N of the products)
constexpr int kRows = 128;   // rows per chunk
constexpr int kAtom = kRows * 128;
constexpr int kPair = 2 * kAtom;
constexpr int kBufs = 3;     // chunks whose rows are known
// Warp 0 looks up rows, warps 1 and 2 load queries (and a pair of FP8MIX rows),
// warp 3 issues products, warps 4-11 take the softmax and fill the tile.  Three
// warps per scheduler leave a thread 168 registers; a thirteenth would leave
// 128, and spills.
constexpr int kSideThreads = 64, kSoftWarp0 = 4, kSoftThreads = 256;
constexpr int kThreads = 32 * kSoftWarp0 + kSoftThreads;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLazy = 14.f;  // log2 headroom before the maximum is raised (fp16 weights reach 2^16)
constexpr int kMaxRope = 64;
constexpr int kMaxSplits = 256;
constexpr int kFewParts = 16;  // fixed split counts up to this are added by one group of threads
constexpr int kMaxNodes = 1184;  // nodes of a call whose units are cut evenly (8 units per SM)
constexpr int kMaxDraft = 1024;
constexpr int kExpMax = 114;     // |e| of a power of two kept beside fp16 values (they reach 2^15 2^114)
constexpr int kRowExpMin = -80;  // e of an FP8MIX row: sums of 2^(s - M) reach 2^30 2^14 2^80
// Below this e the sums take a row's logits again.  At it, P' = 2^(s + e - M) is
// flushed below 2^-126, so s - M < -108, where the row that sets M has s - M >=
// -(65 + 14) (its values are below 2^80, its e up to 65): a loss of 2^-29 of the sum.
constexpr int kRowExpLow = -18;

constexpr int kOffKV = 0;                       // 4 pairs of [128 rows][128 B] atoms: 128 KB
constexpr int kOffQ = kOffKV + 4 * kPair;       // 8 x [64 heads][128 B]: 64 KB
constexpr int kOffP = kOffQ + 8 * kHG * 128;    // [128 rows][128 B]: 16 KB
constexpr int kOffMisc = kOffP + kRows * 128;
// One run of a unit's chunks on one CTA.
struct Segment {
  int bt, hg, c0, c1, nch;
  int64_t slot;  // -1 = the whole unit
};

// A node's rows in order: n_sel entries, n_win window tokens, n_draft drafted
// rows (fewer than 2^31: n_entries < 2^30).
struct NodeRows {
  int vis, n_sel, n_win, n_draft, chunks;
  int64_t win_lo;
};
struct NodeInfo {
  NodeRows rows;
  int64_t win0;  // token of the window's first row
};

struct Misc {
  alignas(16) float mneg[kHG];  // minus the running maximum (0 while there is none)
  alignas(16) float m[kHG];     // running maximum (log2), -inf while there is none
  alignas(16) float corr[kHG];  // rescale factor of a raise; at the end the output factor
  float root[kHG];              // FP8MIX: its square root, as sums may be 2^94 before a raise by 2^150
  float red[4][kHG];        // per-quadrant maxima, then sums
  float cs[2][kMaxRope / 2], sn[2][kMaxRope / 2];  // RoPE at +t (query) and -t (output)
  // of a chunk, the chunk after and the one after that:
  const uint8_t* rowp[kBufs][kRows];               // rows, nullptr where there is none
  int rowe[kBufs][kRows];                          // FP8MIX: the rows' exponents e
  alignas(16) __half scale[kBufs][kRows][8];       // FP8MIX: the rows' seven block scales times 2^-e
  int more[kBufs];          // whether there is such a chunk at all
  int64_t begin, end;       // this CTA's part of the list of chunks
  int node, node_at;        // the node that holds `begin`, and the chunks of it before
  NodeInfo first;           // (kTreeEven) of that node
  int longest;              // > 0: units are cut by themselves into parts of at most so many chunks,
  Segment only;             // and this is the CTA's one
  uint32_t q_top;           // FP8MIX: magnitude bits of the query's largest value
  int some_missing;         // a head has no maximum yet, after the first chunk
  int no_ref;               // a head found no number in the first row
  int dead;                 // a wait ran out: the others do not wait any more
  uint64_t q_full, q_ready, q_empty, kv_full[4], kv_empty[4], s_full, p_full, pv_done, row_full[kBufs], row_empty[kBufs],
      scale_full[kBufs];
  uint32_t tmem_slot;
};
constexpr int kSmemBytes = 1024 + kOffMisc + (int)sizeof(Misc);
static_assert(kSmemBytes <= 227 * 1024, "shared memory");
static_assert(kMaxNodes * sizeof(NodeInfo) <= kOffQ, "the nodes' rows are set up in the row tile");

constexpr int kColO = 0, kColS = 256, kTmemCols = 512;

enum TreeMode { kTreeEven = 0, kTreeWhole = 1, kTreeFixed = 2 };

struct TreePlan {
  int mode, grid, splits;  // splits: kTreeFixed
  int slots;               // partials in the workspace
  int64_t units;
};

struct TreeArgs {
  MqaArgs a;
  TreePlan p;
  int page_shift;  // log2 of the page size, -1 where it is no power of two
};

// Workspace: partial o / l [slot][8 octets of heads][512 dims][8 heads] fp16,
// its scale per dim [slot][512] fp32, (m, l) [slot][64], then (kTreeEven) per
// unit its first slot and their number.
__host__ __device__ __forceinline__ uint4* part_o(const TreePlan&, void* ws, int64_t slot) {
  return static_cast<uint4*>(ws) + slot * (kHG / 8 * kDim);
}
__host__ __device__ __forceinline__ float* part_scale(const TreePlan& p, void* ws, int64_t slot) {
  return reinterpret_cast<float*>(part_o(p, ws, p.slots)) + slot * kDim;
}
__host__ __device__ __forceinline__ float2* part_ml(const TreePlan& p, void* ws, int64_t slot) {
  return reinterpret_cast<float2*>(part_scale(p, ws, p.slots)) + slot * kHG;
}
__host__ __device__ __forceinline__ int2* unit_cut(const TreePlan& p, void* ws) {
  return reinterpret_cast<int2*>(part_ml(p, ws, p.slots));
}
constexpr size_t kSlotBytes = kHG * kDim * 2 + kDim * 4 + kHG * 8;

// x / d, x >= 0 and d >= 1: a 64-bit division (~100 dependent instructions)
// only where the value needs it.
__device__ __noinline__ int64_t div_long(int64_t x, int d) { return x / d; }
__device__ __forceinline__ int64_t div_pos(int64_t x, int d) {
  return (x >> 31) == 0 ? (int64_t)((uint32_t)x / (uint32_t)d) : div_long(x, d);
}

__device__ __noinline__ NodeRows node_rows(const MqaArgs& a, int bt) {
  NodeRows r;
  const int b = bt / a.n_q;
  const int64_t t = a.q_pos[bt], ctx = max64(0, a.ctx_len[b]);
  r.vis = (int)min64(a.n_entries, div_pos(ctx, a.m));
  r.n_sel = a.idx ? a.k : r.vis;
  r.win_lo = max64(0, t - a.window + 1);
  r.n_win = a.window > 0 ? (int)max64(0, min64(t, ctx - 1) - r.win_lo + 1) : 0;
  const int words = (a.n_draft + 31) / 32;
  r.n_draft = 0;
#pragma unroll 1
  for (int w = 0; w < words; ++w) r.n_draft += __popc(tree_word(a, a.tree_mask + (int64_t)bt * words, w));
  r.chunks = (int)((uint32_t)(r.n_sel + r.n_win + r.n_draft + kRows - 1) / kRows);
  if (r.chunks < 1) r.chunks = 1;  // an output of zeros takes a chunk without rows
  if (a.n_nodes != nullptr && bt - b * a.n_q >= a.n_nodes[b]) r.chunks = 0;
  return r;
}
__device__ __forceinline__ NodeInfo node_info(const MqaArgs& a, int bt) {
  return NodeInfo{node_rows(a, bt), a.window > 0 ? a.win_start[bt / a.n_q] : 0};
}
// Addresses of rows p0, p0 + 32, + 64, + 96 of the list, nullptr where absent.
// One warp does this for all of a chunk, so instructions count (with 64-bit
// divisions it took 4,500 cycles): page sizes that are powers of two are
// shifts.  Reads are without conditions, of a place that exists, so that the
// four of a stage are in flight together: behind a chunk's copies each takes
// 1,600 cycles.
__device__ __forceinline__ void rows_at(const TreeArgs& ta, const NodeRows& nr, int bt, int b, int64_t win0, int p0,
                                        int rb, const uint8_t** out) {
  const MqaArgs& a = ta.a;
  int e[4];
  int64_t row[4];
  if (a.idx != nullptr) {
    const int32_t* sel = a.idx + (int64_t)bt * a.k;
#pragma unroll
    for (int i = 0; i < 4; ++i) e[i] = __ldg(sel + min(p0 + 32 * i, a.k - 1));
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) e[i] = p0 + 32 * i;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (p0 + 32 * i >= nr.n_sel || e[i] >= nr.vis) e[i] = -1;
    row[i] = (int64_t)b * a.n_entries + e[i];
  }
  if (a.pages.table != nullptr) {
    const int32_t* table = a.pages.table + (int64_t)b * a.pages.max_pages;
    const int pe = a.pages.page_entries;
    int pg[4], off[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t x = (uint32_t)max(e[i], 0), j = ta.page_shift >= 0 ? x >> ta.page_shift : x / (uint32_t)pe;
      off[i] = (int)(x - j * (uint32_t)pe);
      pg[i] = __ldg(table + j);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      row[i] = (int64_t)pg[i] * pe + off[i];
      if (e[i] >= 0 && (pg[i] < 0 || pg[i] >= a.pages.n_pages)) {
        flag_status(kStatusBadPage);
        e[i] = -1;
      }
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) out[i] = e[i] >= 0 ? static_cast<const uint8_t*>(a.entries) + row[i] * rb : nullptr;
  if (p0 + 96 < nr.n_sel) return;  // entries only
#pragma unroll 1
  for (int i = 0; i < 4; ++i) {
    int p = p0 + 32 * i - nr.n_sel;
    const uint8_t* at = nullptr;
    if (p < 0) continue;
    if (p < nr.n_win) {
      const int64_t w = nr.win_lo + p - win0;
      if (w >= 0 && w < a.win_len) at = static_cast<const uint8_t*>(a.win) + ((int64_t)b * a.win_len + w) * rb;
    } else if ((p -= nr.n_win) < nr.n_draft) {
      at = static_cast<const uint8_t*>(a.draft) +
           ((int64_t)b * a.n_draft + tree_row(a, a.tree_mask + (int64_t)bt * ((a.n_draft + 31) / 32), p)) * rb;
    }
    if (i == 0) out[0] = at;
    if (i == 1) out[1] = at;
    if (i == 2) out[2] = at;
    if (i == 3) out[3] = at;
  }
}

// kTreeEven: equal parts of `total` chunks, none of them empty, the first
// `more` of them one chunk longer.
struct Parts {
  int n, each, more;
  __device__ __forceinline__ Parts(const TreePlan& p, int total)
      : n(min(p.grid, max(total, 1))), each((int)((uint32_t)total / (uint32_t)n)), more(total - each * n) {}
  __device__ __forceinline__ int begin(int i) const { return i * each + min(i, more); }
  // the part that holds chunk x
  __device__ __forceinline__ int of(int x) const {
    const int longer = more * (each + 1);
    return x < longer ? (int)((uint32_t)x / (uint32_t)(each + 1)) : more + (int)((uint32_t)(x - longer) / (uint32_t)each);
  }
};

// The segments of this CTA, in order; every role walks them alike.
struct Walk {
  const TreeArgs& t;
  int64_t pos, end, begin;
  int node, at;  // kTreeEven: the node of pos, and the chunks (parts) of it before pos
  int longest;
  const Misc& ms;
  __device__ __forceinline__ Walk(const TreeArgs& t_, const Misc& ms_) : t(t_), ms(ms_) {
    longest = ms.longest;
    begin = pos = ms.begin;
    end = ms.end;
    node = ms.node;
    at = ms.node_at;
  }
  __device__ __forceinline__ bool next(Segment* s) {
    const int groups = t.a.n_heads / kHG;
    if (longest > 0) {
      if (pos >= end) return false;
      *s = ms.only;
      pos = end;
      return true;
    }
    if (t.p.mode == kTreeEven) {
      while (pos < end) {
        const int nch = node == ms.node ? ms.first.rows.chunks : node_rows(t.a, node).chunks;
        if (at >= nch * groups) {
          ++node;
          at = 0;
          continue;
        }
        s->bt = node;
        s->hg = at >= nch ? 1 : 0;  // one or two groups
        s->c0 = at - s->hg * nch;
        s->c1 = (int)min64(nch, s->c0 + (end - pos));
        s->nch = nch;
        s->slot = s->c0 == 0 && s->c1 == nch ? -1 : 2 * (int64_t)blockIdx.x + (pos == begin ? 0 : 1);
        pos += s->c1 - s->c0;
        at += s->c1 - s->c0;
        return true;
      }
      return false;
    }
    while (pos < end) {
      const int ns = t.p.mode == kTreeFixed ? t.p.splits : 1;
      const int64_t unit = div_pos(pos, ns);
      const int split = (int)(pos - unit * ns);
      s->slot = ns > 1 ? pos : -1;
      pos += t.p.grid;
      s->bt = (int)(groups == 2 ? unit >> 1 : unit);
      s->hg = groups == 2 ? (int)(unit & 1) : 0;
      s->nch = node_rows(t.a, s->bt).chunks;
      if (s->nch == 0) continue;  // the node does not exist
      s->c0 = (int)div_pos((int64_t)split * s->nch, ns);
      s->c1 = (int)div_pos((int64_t)(split + 1) * s->nch, ns);
      return true;
    }
    return false;
  }
};

__device__ __forceinline__ uint8_t* align1024(uint8_t* p) {
  const uint32_t a = smem_u32(p);
  return p + ((1024u - (a & 1023u)) & 1023u);
}
__device__ __forceinline__ uint32_t q_off(int h, int g) {
  return (uint32_t)((g >> 3) * (kHG * 128) + h * 128 + ((((g & 7) ^ (h & 7))) << 4));
}
__device__ __forceinline__ float warp_max_f32(float v) {
  float r;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
  return r;
}
__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
// 2^e, |e| <= 126.
__device__ __forceinline__ float pow2i(int e) { return __uint_as_float((uint32_t)(127 + e) << 23); }
// floor(log2 |x|) of a normal x; -127 for 0 and below the normals, 128 for infinity and NaN.
__device__ __forceinline__ int exponent(float x) { return (int)((__float_as_uint(x) >> 23) & 255u) - 127; }
__device__ __forceinline__ void soft_bar() { asm volatile("bar.sync 1, 256;" ::: "memory"); }
__device__ __forceinline__ bool soft_bar_or(bool v) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbarrier.cta.red.or.pred q, 2, 256, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"((uint32_t)v)
      : "memory");
  return r != 0;
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  uint32_t w;
  memcpy(&w, &h, 4);
  return w;
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  uint32_t w;
  memcpy(&w, &h, 4);
  return w;
}
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool valid) {
  const int n = valid ? 16 : 0;  // 0 bytes read -> 16 zero bytes written
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void prefetch_l2(const void* p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }
// An arrival on the barrier when this thread's earlier cp.async have landed.
__device__ __forceinline__ void cp_async_arrive(uint64_t* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}
__device__ __forceinline__ void st_shared16(uint32_t dst, uint4 v) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(dst), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w)
               : "memory");
}
// mbar_wait for the roles of this kernel: once one wait has run out, all
// others return at once, so the CTA ends within one limit.
__device__ __forceinline__ bool role_wait(Misc& ms, uint64_t* bar, uint32_t parity) {
  if (mbar_try_wait(bar, parity)) return true;
  const unsigned long long t0 = globaltimer_ns();
  for (uint32_t it = 1;; ++it) {
    if (mbar_try_wait(bar, parity)) return true;
    if ((it & 255u) == 0) {
      if (*reinterpret_cast<volatile int*>(&ms.dead) != 0) return false;
      if (globaltimer_ns() - t0 > kWaitTimeoutNs) {
        flag_status(kStatusTimeout);
        *reinterpret_cast<volatile int*>(&ms.dead) = 1;
        return false;
      }
    }
  }
}

// The buffer of a chunk's rows, and the parity of its use.
__device__ __forceinline__ int buf_of(int chunk) { return chunk % kBufs; }
__device__ __forceinline__ uint32_t buf_par(int chunk) { return (uint32_t)(chunk / kBufs) & 1u; }

// Two E4M3 codes as fp16 (exact), times s (each product rounded once).
__device__ __forceinline__ uint32_t decode2(uint32_t codes, __half2 s) {
  const __half2_raw r = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(codes & 0xFFFFu), __NV_E4M3);
  const __half2 v = __hmul2(__half2(r), s);
  uint32_t w;
  memcpy(&w, &v, 4);
  return w;
}

// Sum of each of 32 values over the warp: lane i returns the total of v[i].
__device__ __forceinline__ float reduce32(float* v, int lane) {
#pragma unroll
  for (int d = 16; d >= 1; d >>= 1) {
    const bool up = lane & d;
#pragma unroll
    for (int i = 0; i < d; ++i) {
      const float keep = up ? v[i + d] : v[i], give = up ? v[i] : v[i + d];
      v[i] = keep + __shfl_xor_sync(0xffffffffu, give, d);
    }
  }
  return v[0];
}

// ------------------------------------------------------------ filling the tile
// BF16 rows come by cp.async (2,000 cycles per 128 KB on all SMs at once, 66
// B/cycle/SM): a 16-byte piece g of the 256 bytes that a pair has of a row, rows
// t / 16, + 16, ...  All addresses are in registers before the first copy: a
// shared-memory read before each made them take three times as long to issue.
// FP8MIX rows go through registers: the softmax threads take pairs 0-2 (16 codes of a row a piece: dims 128 p + 16 g ..; rows t / 8,
// + 32, ...), the row warps pair 3, 64 codes and the 64 bf16.
struct F8Pair {
  static constexpr int kPieces = kRows / 32;
  uint4 v[kPieces];
  __device__ __forceinline__ void load(const Misc& ms, int t, int buf, int p) {
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      const uint8_t* src = ms.rowp[buf][(t >> 3) + 32 * i];
      v[i] = src != nullptr ? __ldcg(reinterpret_cast<const uint4*>(src + 128 * p + 16 * (t & 7))) : make_uint4(0, 0, 0, 0);
    }
  }
  // 16-byte units 2 g and 2 g + 1 of the pair's 16, block scale 2 p + g / 4.
  // Lanes of the second atom store their odd unit first: the eight lanes of a
  // row then meet eight different banks (two by two on four otherwise).
  __device__ __forceinline__ void store(const Misc& ms, uint32_t kv, int t, int buf, int p) const {
    const int g = t & 7, r0 = t >> 3, odd = g >> 2, q = 2 * (g & 3);
    const uint32_t at0 = kv + p * kPair + odd * kAtom + r0 * 128;
    const uint32_t first = (uint32_t)(((q + odd) ^ (r0 & 7)) << 4), second = (uint32_t)(((q + 1 - odd) ^ (r0 & 7)) << 4);
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      const __half2 s = __half2half2(ms.scale[buf][r0 + 32 * i][2 * p + odd]);
      const uint32_t at = at0 + i * 4096;
      const uint2 lo = make_uint2(v[i].x, v[i].y), hi = make_uint2(v[i].z, v[i].w);
      const uint2 a = odd ? hi : lo, b = odd ? lo : hi;
      st_shared16(at + first, make_uint4(decode2(a.x, s), decode2(a.x >> 16, s), decode2(a.y, s), decode2(a.y >> 16, s)));
      st_shared16(at + second, make_uint4(decode2(b.x, s), decode2(b.x >> 16, s), decode2(b.y, s), decode2(b.y >> 16, s)));
    }
  }
};
// Pair 3: a row's 12 pieces of 16 bytes (from byte 384), four of codes and
// eight of bf16, and its scales; threads t of 64 take pieces t % 4 + 4 j and
// scales 2 (t % 4), + 1 of rows t / 4, + 16, ...
struct F8Last {
  static constexpr int kPieces = kRows / 32;  // of half of the rows
  uint4 v[3][kPieces], more[kPieces];
  __device__ __forceinline__ static const uint8_t* row(const Misc& ms, int t, int buf, int i) {
    return ms.rowp[buf][(t >> 2) + 16 * i];
  }
  __device__ __forceinline__ static uint4 piece(const uint8_t* src, int t, int j) {
    return src != nullptr ? __ldcg(reinterpret_cast<const uint4*>(src + 384 + 64 * j + 16 * (t & 3)))
                          : make_uint4(0, 0, 0, 0);
  }
  __device__ __forceinline__ void load(const Misc& ms, int t, int buf, int half) {
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      const uint8_t* src = row(ms, t, buf, kPieces * half + i);
#pragma unroll
      for (int j = 0; j < 3; ++j) v[j][i] = piece(src, t, j);
    }
  }
  // the rows' exponents and scales times 2^-e
  __device__ __forceinline__ static void scales(Misc& ms, int t, int buf) {
    const int g = t & 3;
#pragma unroll 1
    for (int half = 0; half < 2; ++half) {
      uint4 u[2][kPieces];
      float2 sc[kPieces];
#pragma unroll
      for (int i = 0; i < kPieces; ++i) {
        const uint8_t* src = row(ms, t, buf, kPieces * half + i);
        u[0][i] = piece(src, t, 1);
        u[1][i] = piece(src, t, 2);
        sc[i] = src != nullptr ? __ldcg(reinterpret_cast<const float2*>(src + 576 + 8 * g)) : make_float2(0.f, 0.f);
      }
#pragma unroll
      for (int i = 0; i < kPieces; ++i) {
        const int r = (t >> 2) + 16 * (kPieces * half + i);
        if (g == 3) sc[i].y = 0.f;  // padding
        uint32_t top = 0;  // the largest magnitude bits of the bf16, two at a time
#pragma unroll
        for (int j = 0; j < 2; ++j)
          top = __vmaxu2(top, __vmaxu2(__vmaxu2(u[j][i].x & 0x7FFF7FFFu, u[j][i].y & 0x7FFF7FFFu),
                                       __vmaxu2(u[j][i].z & 0x7FFF7FFFu, u[j][i].w & 0x7FFF7FFFu)));
        const float tail = fmaxf(__uint_as_float(top << 16), __uint_as_float(top & 0xFFFF0000u));
        // codes reach 448 < 2^9: scales below 2^7 and bf16 values below 2^16 fit fp16
        int e = max(exponent(fmaxf(fabsf(sc[i].x), fabsf(sc[i].y))) + 1 - 7, exponent(tail) + 1 - 15);
        e = max(e, __shfl_xor_sync(0xffffffffu, e, 1));
        e = max(e, __shfl_xor_sync(0xffffffffu, e, 2));
        e = max(kRowExpMin, min(kExpMax, e));
        const float f = pow2i(-e);
        *reinterpret_cast<uint32_t*>(&ms.scale[buf][r][2 * g]) = pack_f16(sc[i].x * f, sc[i].y * f);
        if (g == 0) ms.rowe[buf][r] = e;
      }
    }
  }
  // everything as fp16: the codes' 16 values into v[0] and `more`, the bf16 in place
  __device__ __forceinline__ void decode(const Misc& ms, int t, int buf, int half) {
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      const int r = (t >> 2) + 16 * (kPieces * half + i);
      const __half2 s = __half2half2(ms.scale[buf][r][6]);
      const uint4 c = v[0][i];
      v[0][i] = make_uint4(decode2(c.x, s), decode2(c.x >> 16, s), decode2(c.y, s), decode2(c.y >> 16, s));
      more[i] = make_uint4(decode2(c.z, s), decode2(c.z >> 16, s), decode2(c.w, s), decode2(c.w >> 16, s));
      const float f = pow2i(-ms.rowe[buf][r]);
#pragma unroll
      for (int j = 1; j < 3; ++j) {
        uint32_t w[4] = {v[j][i].x, v[j][i].y, v[j][i].z, v[j][i].w};
#pragma unroll
        for (int q = 0; q < 4; ++q)
          w[q] = pack_f16(__uint_as_float(w[q] << 16) * f, __uint_as_float(w[q] & 0xFFFF0000u) * f);
        v[j][i] = make_uint4(w[0], w[1], w[2], w[3]);
      }
    }
  }
  __device__ __forceinline__ void store(uint32_t kv, int t, int half) const {
    const int g = t & 3, x = (t >> 2) & 7;
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      const uint32_t at = kv + 3 * kPair + ((t >> 2) + 16 * (kPieces * half + i)) * 128;
      st_shared16(at + (((2 * g) ^ x) << 4), v[0][i]);
      st_shared16(at + (((2 * g + 1) ^ x) << 4), more[i]);
#pragma unroll
      for (int j = 1; j < 3; ++j) st_shared16(at + kAtom + (((4 * (j - 1) + g) ^ x) << 4), v[j][i]);
    }
  }
};

// The softmax threads' part of filling the tile.
template <bool FP8>
struct Filler;
template <>
struct Filler<false> {
  __device__ __forceinline__ void start(const Misc&, int, int) {}
  // chunk `chunk`, pair by pair as the products of the chunk before have read them
  __device__ __forceinline__ void finish(Misc& ms, uint32_t kv, int st, int chunk, const void* dummy) {
    constexpr int kPieces = kRows / 16;
    const int g = st & 15, r0 = st >> 4, buf = buf_of(chunk);
    const uint8_t* src[kPieces];
    uint32_t there = 0;
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      src[i] = ms.rowp[buf][r0 + 16 * i];
      there |= (src[i] != nullptr ? 1u : 0u) << i;
      src[i] = src[i] != nullptr ? src[i] + g * 16 : static_cast<const uint8_t*>(dummy);
    }
    const uint32_t dst0 = kv + (g >> 3) * kAtom + r0 * 128 + (((g & 7) ^ (r0 & 7)) << 4);
#pragma unroll 1
    for (int p = 0; p < 4; ++p) {
      if (chunk > 0) role_wait(ms, &ms.kv_empty[p], (chunk - 1) & 1);
#pragma unroll
      for (int i = 0; i < kPieces; ++i) {
        const bool on = (there >> i) & 1u;
        cp_async16(dst0 + p * kPair + i * 2048, on ? src[i] + p * 256 : src[i], on);
      }
      cp_async_arrive(&ms.kv_full[p]);
    }
  }
};
template <>
struct Filler<true> {
  F8Pair pair, next, last;
  // the three pairs on their way to registers (the sums of the chunk before are taken meanwhile)
  __device__ __forceinline__ void start(const Misc& ms, int st, int chunk) {
    const int buf = buf_of(chunk);
    pair.load(ms, st, buf, 0);
    next.load(ms, st, buf, 1);
    last.load(ms, st, buf, 2);
  }
  __device__ __forceinline__ void finish(Misc& ms, uint32_t kv, int st, int chunk, const void*) {
    const int buf = buf_of(chunk);
    role_wait(ms, &ms.scale_full[buf], buf_par(chunk));
    // one body for all pairs: the roles' loops over chunks together overflow
    // the instruction cache as it is
#pragma unroll 1
    for (int p = 0; p < 3; ++p) {
      if (chunk > 0) role_wait(ms, &ms.kv_empty[p], (chunk - 1) & 1);
      pair.store(ms, kv, st, buf, p);
      fence_proxy_async_smem();
      mbar_arrive(&ms.kv_full[p]);
      pair = next;
      next = last;
    }
  }
};

// The query rows of the unit in place: RMSNorm and RoPE with the arithmetic
// and order of csa_rmsnorm_rope.
__device__ __forceinline__ void turn_query(const MqaArgs& a, const Misc& ms, uint8_t* Qs, int st, int lane) {
  const int d_rope = kDim - a.q_rope_dims;
#pragma unroll 1
  for (int h = st >> 5; h < kHG; h += kSoftThreads / 32) {
    float v[2][8];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const uint4 u = *reinterpret_cast<const uint4*>(Qs + q_off(h, lane + 32 * k));
      const uint32_t w4[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        v[k][2 * j] = __uint_as_float(w4[j] << 16);
        v[k][2 * j + 1] = __uint_as_float(w4[j] & 0xFFFF0000u);
      }
    }
    if (a.q_norm_g != nullptr) {
      float ss = 0.f;
#pragma unroll
      for (int k = 0; k < 2; ++k)
#pragma unroll
        for (int q = 0; q < 8; ++q) ss = fmaf(v[k][q], v[k][q], ss);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
      const float inv = rms_inv(ss, kDim, a.q_norm_eps);
#pragma unroll
      for (int k = 0; k < 2; ++k)
#pragma unroll
        for (int q = 0; q < 8; ++q) v[k][q] = __fmul_rn(__fmul_rn(v[k][q], inv), a.q_norm_g[8 * (lane + 32 * k) + q]);
    }
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int d0 = 8 * (lane + 32 * k);
      if (a.q_rope_dims > 0 && d0 >= d_rope) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int kp = (d0 - d_rope) / 2 + j;
          rope_turn(v[k][2 * j], v[k][2 * j + 1], ms.cs[0][kp], ms.sn[0][kp]);
        }
      }
      *reinterpret_cast<uint4*>(Qs + q_off(h, lane + 32 * k)) =
          make_uint4(pack_bf16(v[k][0], v[k][1]), pack_bf16(v[k][2], v[k][3]), pack_bf16(v[k][4], v[k][5]),
                     pack_bf16(v[k][6], v[k][7]));
    }
  }
}

// For FP8MIX rows: the unit's query as fp16 times a power of two that puts its
// largest finite value below 2^15 (values down to 2^-29 of it keep their 8 bits;
// below, a logit is off by no more than 2^-39 of the largest there can be).
// Returns the power that the logits are to be multiplied by.
__device__ __forceinline__ float query_to_f16(Misc& ms, uint8_t* Qs, int st, int lane) {
  constexpr int kPieces = kHG * kDim / 8 / kSoftThreads;
  uint4* q = reinterpret_cast<uint4*>(Qs) + st;
  // magnitude bits of the largest value, two at a time; with `limit` only of those below it
  const auto largest = [&](bool limit) {
    uint32_t top = 0;
    const auto mag = [&](uint32_t w) {
      w &= 0x7FFF7FFFu;
      return limit ? w & __vcmpltu2(w, 0x7F807F80u) : w;
    };
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      const uint4 u = q[i * kSoftThreads];
      top = __vmaxu2(top, __vmaxu2(__vmaxu2(mag(u.x), mag(u.y)), __vmaxu2(mag(u.z), mag(u.w))));
    }
    top = __reduce_max_sync(0xffffffffu, max(top & 0xFFFFu, top >> 16));
    if (lane == 0) atomicMax(&ms.q_top, top);
    soft_bar();
    return ms.q_top;
  };
  uint32_t top = largest(false);
  if (top >= 0x7F80u) {  // a head with an infinity or a NaN, which the others shall not feel
    soft_bar();
    if (st == 0) ms.q_top = 0;
    soft_bar();
    top = largest(true);
  }
  const int e = max(-kExpMax, min(kExpMax, exponent(__uint_as_float(top << 16)) - 14));
  const float f = pow2i(-e);
#pragma unroll
  for (int i = 0; i < kPieces; ++i) {
    const uint4 u = q[i * kSoftThreads];
    uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int j = 0; j < 4; ++j)
      w[j] = pack_f16(__uint_as_float(w[j] << 16) * f, __uint_as_float(w[j] & 0xFFFF0000u) * f);
    q[i * kSoftThreads] = make_uint4(w[0], w[1], w[2], w[3]);
  }
  return pow2i(e);
}

template <bool FP8>
__global__ void __launch_bounds__(kThreads, 1)
    tree_umma_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ TreeArgs ta) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* base = align1024(smem_raw);
  uint8_t* KV = base + kOffKV;
  uint8_t* Qs = base + kOffQ;
  uint8_t* Ps = base + kOffP;
  Misc& ms = *reinterpret_cast<Misc*>(base + kOffMisc);
  const MqaArgs& a = ta.a;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int groups = a.n_heads / kHG;

  if (tid == 0) {
    ms.dead = 0;
    mbar_init(&ms.q_full, 1);
    mbar_init(&ms.q_ready, 1);
    mbar_init(&ms.q_empty, 1);
    for (int i = 0; i < 4; ++i) {
      mbar_init(&ms.kv_full[i], FP8 && i == 3 ? kSideThreads : kSoftThreads);
      mbar_init(&ms.kv_empty[i], 1);
    }
    mbar_init(&ms.s_full, 1);
    mbar_init(&ms.p_full, 1);
    mbar_init(&ms.pv_done, 1);
    for (int i = 0; i < kBufs; ++i) {
      mbar_init(&ms.row_full[i], 1);
      mbar_init(&ms.row_empty[i], 1);
      mbar_init(&ms.scale_full[i], kSideThreads);
    }
    fence_barrier_init();
  }
  // whoever stops waiting finds an address that may be read
  for (int i = tid; i < kBufs * kRows; i += kThreads) (&ms.rowp[0][0])[i] = nullptr;
  if (tid < kBufs) ms.more[tid] = 0;
  if (warp == kSoftWarp0 - 1) tmem_alloc(&ms.tmem_slot, kTmemCols);
  after_previous();
  int total = 0;
  if (ta.p.mode == kTreeEven) {
    // what is known of every node, in the row tile; one warp sums the chunks
    // and finds where this CTA's part begins
    NodeInfo* info = reinterpret_cast<NodeInfo*>(KV);
    const int nodes = a.batch * a.n_q;
#pragma unroll 1
    for (int n = tid; n < nodes; n += kThreads) info[n] = node_info(a, n);
    __syncthreads();
    if (warp == 0) {
      int sum = 0;
#pragma unroll 1
      for (int n = lane; n < nodes; n += 32) sum += info[n].rows.chunks;
      total = __reduce_add_sync(0xffffffffu, sum) * groups;
      // A CTA that passes from one unit to the next pays about as much as for
      // two chunks (output, sums, a new query).  So units are cut by themselves,
      // each part on a CTA of its own, if that makes the longest part at most
      // two chunks longer: 64 units of 10 chunks took 53 us in 148 equal parts
      // and 36 us in 128 halves; units of one part need no combine kernel.
      const Parts parts(ta.p, total);
      const int t0 = parts.each + (parts.more > 0);
      int n_cut[3] = {0, 0, 0};
#pragma unroll 1
      for (int n = lane; total > 0 && n < nodes; n += 32)
#pragma unroll
        for (int i = 0; i < 3; ++i)
          n_cut[i] += (int)((uint32_t)(info[n].rows.chunks + t0 + i - 1) / (uint32_t)(t0 + i));
      int longest = 0;
#pragma unroll
      for (int i = 2; i >= 0; --i)
        if (__reduce_add_sync(0xffffffffu, n_cut[i]) * groups <= ta.p.grid && total > 0) longest = t0 + i;
      // the part, or its first chunk
      const int begin = longest > 0 ? blockIdx.x : blockIdx.x < parts.n ? parts.begin(blockIdx.x) : 0;
      int end = longest > 0 || blockIdx.x >= parts.n ? 0 : parts.begin(blockIdx.x + 1);
      int run = 0;  // chunks (parts) of the nodes before n0
      int node = 0, node_at = 0;
#pragma unroll 1
      for (int n0 = 0; n0 < nodes; n0 += 32) {
        int mine = n0 + lane < nodes ? info[n0 + lane].rows.chunks : 0;
        if (longest > 0) mine = (int)((uint32_t)(mine + longest - 1) / (uint32_t)longest);
        mine *= groups;
        int inc = mine;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
          const int o = __shfl_up_sync(0xffffffffu, inc, d);
          if (lane >= d) inc += o;
        }
        const int first = run + inc - mine;
        const uint32_t who = __ballot_sync(0xffffffffu, first <= begin && begin < run + inc);
        if (who != 0) {
          node = n0 + __ffs(who) - 1;
          node_at = begin - __shfl_sync(0xffffffffu, first, __ffs(who) - 1);
          if (longest > 0) end = begin + 1;
          break;
        }
        run += __shfl_sync(0xffffffffu, inc, 31);
      }
      if (lane == 0) {
        ms.begin = begin;
        ms.end = end;
        ms.node = node;
        ms.node_at = node_at;
        ms.longest = longest;
        ms.first = info[node];
        if (longest > 0 && end > 0) {
          const int nch = info[node].rows.chunks, n_parts = (int)((uint32_t)(nch + longest - 1) / (uint32_t)longest);
          const int hg = node_at >= n_parts ? 1 : 0, part = node_at - hg * n_parts;  // one or two groups
          ms.only = Segment{node, hg, (int)((uint32_t)(part * nch) / (uint32_t)n_parts),
                            (int)((uint32_t)((part + 1) * nch) / (uint32_t)n_parts), nch,
                            n_parts == 1 ? -1 : (int64_t)blockIdx.x};
          // where the unit's parts are, for the combine kernel (next to one another)
          if (part == 0)
            unit_cut(ta.p, a.ws)[node * groups + hg] = n_parts > 1 ? make_int2(blockIdx.x, -n_parts) : make_int2(0, 0);
        }
      }
    }
  } else if (tid == 0) {
    ms.longest = 0;
    ms.begin = blockIdx.x;
    ms.end = ta.p.units * (ta.p.mode == kTreeFixed ? ta.p.splits : 1);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = ms.tmem_slot;
  const bool turn_q = FP8 || a.q_norm_g != nullptr || a.q_rope_dims > 0;

  if (warp == 0) {
    // ------------------------------------------------------------ rows
    // Up to three chunks ahead: an address is two or three dependent reads away.
    Walk walk(ta, ms);
    Segment s;
    int chunk = 0;
    const int rb = (int)row_bytes(a.kv_dt, kDim);
    while (walk.next(&s)) {
      const int b = s.bt / a.n_q;
      const NodeInfo ni = ta.p.mode == kTreeEven && s.bt == ms.node ? ms.first : node_info(a, s.bt);
      if (lane == 0 && ta.p.mode == kTreeEven && walk.longest == 0 && s.c0 == 0) {
        // where the parts cut this unit, for the combine kernel
        int2 cut = make_int2(0, 0);
        if (s.c1 < s.nch)
          cut = make_int2((int)s.slot, Parts(ta.p, total).of((int)walk.pos - s.c1 + s.nch - 1) - (int)blockIdx.x + 1);
        unit_cut(ta.p, a.ws)[s.bt * groups + s.hg] = cut;
      }
      for (int c = s.c0; c < s.c1; ++c, ++chunk) {
        const int buf = buf_of(chunk);
        const uint8_t* p[4];
        rows_at(ta, ni.rows, s.bt, b, ni.win0, c * kRows + lane, rb, p);
        if (chunk >= kBufs) role_wait(ms, &ms.row_empty[buf], buf_par(chunk) ^ 1u);
#pragma unroll
        for (int i = 0; i < 4; ++i) ms.rowp[buf][lane + 32 * i] = p[i];
        ms.more[buf] = 1;
        __syncwarp();
        if (lane == 0) mbar_arrive(&ms.row_full[buf]);
        if (FP8 && chunk > 0) {
          // on their way to L2 already, as their loads wait for registers until
          // the softmax is done (CSA at 1M 48.7 -> 46.6 us; BF16 rows, copied
          // as their places become free, lose by it: HCA at 1M 187 -> 197)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (p[i] != nullptr)
              for (int at = 0; at < rb; at += 128) prefetch_l2(p[i] + at);
        }
      }
    }
    // no more chunks
    if (chunk >= kBufs) role_wait(ms, &ms.row_empty[buf_of(chunk)], buf_par(chunk) ^ 1u);
    ms.more[buf_of(chunk)] = 0;
    __syncwarp();
    if (lane == 0) mbar_arrive(&ms.row_full[buf_of(chunk)]);
  } else if (warp < 3) {
    // ------------------------------------------------------------ queries, FP8MIX pair 3
    Walk walk(ta, ms);
    Segment s;
    int chunk = 0, seg = 0;
    while ((FP8 || warp == 1) && walk.next(&s)) {
      if (s.c0 == s.c1) continue;
      if (tid == 32) {
        if (seg > 0) role_wait(ms, &ms.q_empty, (seg - 1) & 1);
        mbar_arrive_expect_tx(&ms.q_full, kHG * kDim * 2);
        const int qrow = s.bt * a.n_heads + s.hg * kHG;
        for (int at = 0; at < 8; ++at) tma_load_2d(Qs + at * (kHG * 128), &tmQ, &ms.q_full, 64 * at, qrow);
      }
      __syncwarp();
      ++seg;
      if (FP8) {
        for (int c = s.c0; c < s.c1; ++c, ++chunk) {
          const int buf = buf_of(chunk), t = tid - 32;
          F8Last last;
          role_wait(ms, &ms.row_full[buf], buf_par(chunk));
          F8Last::scales(ms, t, buf);
          mbar_arrive(&ms.scale_full[buf]);
          __syncwarp();  // (a row's scales are made and used within a warp)
#pragma unroll 1
          for (int half = 0; half < 2; ++half) {
            last.load(ms, t, buf, half);
            last.decode(ms, t, buf, half);  // the first half ahead of the wait for the pair's place
            if (chunk > 0 && half == 0) role_wait(ms, &ms.kv_empty[3], (chunk - 1) & 1);
            last.store(smem_u32(KV), t, half);
          }
          fence_proxy_async_smem();
          mbar_arrive(&ms.kv_full[3]);
        }
      }
    }
  } else if (warp == kSoftWarp0 - 1) {
    // ------------------------------------------------------------ products
    Walk walk(ta, ms);
    Segment s;
    int chunk = 0, seg = 0;  // seg: segments with chunks
    constexpr uint32_t kFmt = FP8 ? (1u << 7) | (1u << 10) : 0u;  // bf16 operands, or fp16 (0) for decoded rows
    constexpr uint32_t kIdescQK = idesc_bf16_f32(128, kHG) & ~kFmt;
    constexpr uint32_t kIdescPV = idesc_bf16_f32_major(128, kHG, 1, 1) & ~kFmt;
    // descriptors advance by a step's bytes / 16 in their low word
    const uint64_t kd = umma_desc_sw128(smem_u32(KV)), qd = umma_desc_sw128(smem_u32(Qs)),
                   vd = umma_desc_sw128_mn(smem_u32(KV), kAtom, 1024), pd = umma_desc_sw128_mn(smem_u32(Ps), kAtom, 1024);
    if (elect_one()) {
      bool ok = true;
      while (ok && walk.next(&s)) {
        for (int c = s.c0; ok && c < s.c1; ++c, ++chunk) {
          const uint32_t par = chunk & 1;
          if (c == s.c0) ok = role_wait(ms, turn_q ? &ms.q_ready : &ms.q_full, seg & 1);
#pragma unroll(FP8 ? 1 : 4)
          for (int p = 0; p < 4; ++p) {
            ok = ok && role_wait(ms, &ms.kv_full[p], par);
            if (!ok) break;
            if (!FP8) fence_proxy_async_smem();  // the rows were written by cp.async
            tc_fence_after();
#pragma unroll
            for (int kk = 0; kk < 8; ++kk)
              tc_mma_f16(tmem + kColS, kd + (uint64_t)(p * (kPair / 16) + (kk >> 2) * (kAtom / 16) + 2 * (kk & 3)),
                         qd + (uint64_t)((2 * p + (kk >> 2)) * (kHG * 128 / 16) + 2 * (kk & 3)), kIdescQK,
                         p + kk > 0 ? 1u : 0u);
          }
          if (!ok) break;
          tc_commit(&ms.s_full);
          if (c + 1 == s.c1) tc_commit(&ms.q_empty);
          ok = role_wait(ms, &ms.p_full, par);
          if (!ok) break;
          tc_fence_after();
          const uint32_t add = c > s.c0 ? 1u : 0u;
#pragma unroll(FP8 ? 1 : 4)
          for (int p = 0; p < 4; ++p) {
#pragma unroll
            for (int kk = 0; kk < kRows / 16; ++kk)
              tc_mma_f16(tmem + kColO + p * kHG, vd + (uint64_t)(p * (kPair / 16) + 128 * kk),
                         pd + (uint64_t)(128 * kk), kIdescPV, kk > 0 ? 1u : add);
            tc_commit(&ms.kv_empty[p]);
          }
          tc_commit(&ms.pv_done);
        }
        if (s.c0 < s.c1) ++seg;
      }
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------ softmax
    const int st = tid - 32 * kSoftWarp0;                        // 0..255
    const int quad = warp & 3, half = (warp - kSoftWarp0) >> 2;  // rows 32 quad .., heads 32 half ..
    const int row = 32 * quad + lane;
    const uint32_t lane_base = (uint32_t)(32 * quad) << 16;
    const uint32_t prow = smem_u32(Ps) + row * 128, kv = smem_u32(KV);
    float sl2 = a.scale * kLog2e;
    const float4* mneg = reinterpret_cast<const float4*>(ms.mneg + 32 * half);
    Walk walk(ta, ms);
    Segment s;
    int chunk = 0, seg = 0;
    Filler<FP8> filler;
    role_wait(ms, &ms.row_full[0], 0);
    if (!turn_q && ms.more[0] != 0) filler.finish(ms, kv, st, 0, a.Q);
    while (walk.next(&s)) {
      if (st < kHG) {
        ms.m[st] = -INFINITY;
        ms.mneg[st] = 0.f;
      }
      if (st == 0) {
        ms.some_missing = 0;
        ms.no_ref = 0;
        ms.q_top = 0;
      }
      if (st < 32 && a.q_rope_dims + a.out_rope_dims > 0) {
        const int64_t t = a.q_pos[s.bt];
        if (st < a.q_rope_dims / 2)
          rope_sincos((double)t, rope_theta(a.rope_base, st, a.q_rope_dims), &ms.sn[0][st], &ms.cs[0][st]);
        if (st < a.out_rope_dims / 2)
          rope_sincos((double)t * -1.0, rope_theta(a.rope_base, st, a.out_rope_dims), &ms.sn[1][st], &ms.cs[1][st]);
      }
      soft_bar();
      if (turn_q && s.c0 < s.c1) {
        role_wait(ms, &ms.q_full, seg & 1);
        if (a.q_norm_g != nullptr || a.q_rope_dims > 0) {
          turn_query(a, ms, Qs, st, lane);
          if (FP8) soft_bar();
        }
        if (FP8) sl2 = a.scale * kLog2e * query_to_f16(ms, Qs, st, lane);
        fence_proxy_async_smem();
        soft_bar();
        if (st == 0) mbar_arrive(&ms.q_ready);
        if (chunk == 0) {
          filler.start(ms, st, 0);
          filler.finish(ms, kv, st, 0, a.Q);
        }
      }
      if (s.c0 < s.c1) ++seg;
      // sums of the weights: of this thread's row in 32 heads; for FP8MIX rows,
      // whose loads want the registers, of the warp's rows in the lane's head
      float l[FP8 ? 1 : 32];
#pragma unroll
      for (int h = 0; h < (FP8 ? 1 : 32); ++h) l[h] = 0.f;
      for (int c = s.c0; c < s.c1; ++c, ++chunk) {
        const uint32_t par = chunk & 1;
        const int buf = buf_of(chunk);
        const bool on = ms.rowp[buf][row] != nullptr;
        const int e = FP8 && on ? ms.rowe[buf][row] : 0;
        const float sc = FP8 ? sl2 * pow2i(e) : sl2, er = (float)e;
        role_wait(ms, &ms.s_full, par);
        tc_fence_after();
        // the products of the chunk before have read P
        if (chunk > 0) role_wait(ms, &ms.pv_done, par ^ 1u);
        float x[32];  // S, then the weights
        const auto logits = [&]() {
          tmem_ld_32x32b_x32(tmem + lane_base + kColS + 32 * half, x);
          tmem_ld_wait();
        };
        bool above = ms.some_missing != 0;
        if (c == s.c0) {
          // the unit's first chunk: the logits of the first row of quadrant 0
          // will do for maxima, as the vote raises what is too low (the maxima
          // of 128 rows by warp reductions took 1,500 cycles)
          if (quad == 0) {
            logits();
            const uint32_t who = __ballot_sync(0xffffffffu, on);
            bool fine = who != 0;
            if (lane == __ffs(who) - 1) {
#pragma unroll
              for (int g = 0; g < 8; ++g) {
                float w[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                  w[i] = FP8 ? fmaf(x[4 * g + i], sc, er) : x[4 * g + i] * sc;
                  fine = fine && fabsf(w[i]) < INFINITY;
                }
                reinterpret_cast<float4*>(ms.m + 32 * half)[g] = make_float4(w[0], w[1], w[2], w[3]);
                reinterpret_cast<float4*>(ms.mneg + 32 * half)[g] = make_float4(-w[0], -w[1], -w[2], -w[3]);
              }
            }
            if (!__all_sync(0xffffffffu, fine) && lane == 0) ms.no_ref = 1;
          }
          soft_bar();
          above = ms.no_ref != 0;
        }
        for (int round = 0;; ++round) {
          if (round > 0 || !above) {
            above = false;
            logits();
#pragma unroll
            for (int g = 0; g < 8; ++g) {
              const float4 mn = mneg[g];
              const float m4[4] = {mn.x, mn.y, mn.z, mn.w};
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const float w = fmaf(x[4 * g + i], sc, FP8 ? er + m4[i] : m4[i]);
                const float v = on ? w : -INFINITY;
                above |= v > kLazy;
                x[4 * g + i] = ex2(v);
              }
            }
#pragma unroll
            for (int g = 0; g < 4; ++g) {
              uint32_t w[4];
#pragma unroll
              for (int i = 0; i < 4; ++i)
                w[i] = FP8 ? pack_f16(x[8 * g + 2 * i], x[8 * g + 2 * i + 1])
                           : pack_bf16(x[8 * g + 2 * i], x[8 * g + 2 * i + 1]);
              st_shared16(prow + (((4 * half + g) ^ (row & 7)) << 4), make_uint4(w[0], w[1], w[2], w[3]));
            }
            tc_fence_before();
            fence_proxy_async_smem();
          }
          if (!soft_bar_or(above) || round > 0) break;
          // the maxima of this chunk, and the raise; then P against the new ones
          logits();
#pragma unroll
          for (int h = 0; h < 32; ++h) {
            const float wm = warp_max_f32(on ? (FP8 ? fmaf(x[h], sc, er) : x[h] * sc) : -INFINITY);
            if (lane == h) ms.red[quad][32 * half + h] = wm;
          }
          soft_bar();
          if (st < kHG) {
            const float cm = fmaxf(fmaxf(ms.red[0][st], ms.red[1][st]), fmaxf(ms.red[2][st], ms.red[3][st]));
            const float old = ms.m[st];
            const float m = cm > old + kLazy || old == -INFINITY ? fmaxf(cm, old) : old;  // (a NaN stays)
            const float down = old == -INFINITY || m == old ? 0.f : old - m;
            ms.corr[st] = exp2f(down);
            if (FP8) ms.root[st] = exp2f(0.5f * down);
            ms.m[st] = m;
            ms.mneg[st] = m == -INFINITY ? 0.f : -m;
          }
          if (st == 0) ms.some_missing = 0;
          soft_bar();
          if (st < kHG && ms.m[st] == -INFINITY) ms.some_missing = 1;
          if (c > s.c0) {
            // sums and O^T so far (lane = dim; this warp's two slabs)
#pragma unroll
            for (int h = 0; h < (FP8 ? 1 : 32); ++h) {
              const float r = FP8 ? ms.root[32 * half + lane] : ms.corr[32 * half + h];
              l[h] *= r;
              if (FP8) l[h] *= r;
            }
            tc_fence_after();
#pragma unroll 1
            for (int q = 0; q < 4; ++q) {
              const uint32_t col = tmem + lane_base + kColO + (2 * half + (q >> 1)) * kHG + 32 * (q & 1);
              tmem_ld_32x32b_x32(col, x);
              tmem_ld_wait();
#pragma unroll
              for (int h = 0; h < 32; ++h) x[h] *= ms.corr[32 * (q & 1) + h];
              tmem_st_32x32b_x32(col, x);
            }
            tmem_st_wait();
          }
        }
        if (st == 0) {
          mbar_arrive(&ms.p_full);
          mbar_arrive(&ms.row_empty[buf]);
        }
        float back = FP8 ? pow2i(-e) : 1.f;
        if (FP8 && __any_sync(0xffffffffu, e < kRowExpLow)) {
          logits();  // they are there until all softmax warps have filled the tile
          tc_fence_before();
          back = 1.f;
#pragma unroll
          for (int g = 0; g < 8; ++g) {
            const float4 mn = mneg[g];
            const float m4[4] = {mn.x, mn.y, mn.z, mn.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) x[4 * g + i] = on ? ex2(fmaf(x[4 * g + i], sc, m4[i])) : 0.f;
          }
        }
        // the next chunk, if there is one, into the tile
        role_wait(ms, &ms.row_full[buf_of(chunk + 1)], buf_par(chunk + 1));
        const bool more = ms.more[buf_of(chunk + 1)] != 0;
        if (more) filler.start(ms, st, chunk + 1);
        if (FP8) {
#pragma unroll
          for (int h = 0; h < 32; ++h) x[h] *= back;
          l[0] += reduce32(x, lane);
        } else {
#pragma unroll
          for (int h = 0; h < 32; ++h) l[FP8 ? 0 : h] += x[h];
        }
        if (more) filler.finish(ms, kv, st, chunk + 1, a.Q);
      }
      // ---- the unit's (or part's) sums and output
      ms.red[quad][32 * half + lane] = FP8 ? l[0] : reduce32(l, lane);
      soft_bar();
      if (st < kHG) {
        const float L = (ms.red[0][st] + ms.red[1][st]) + (ms.red[2][st] + ms.red[3][st]);
        const float m = ms.m[st];
        float f = 0.f;
        if (s.slot >= 0) {
          part_ml(ta.p, a.ws, s.slot)[st] = make_float2(m, L);
          if (m != -INFINITY) f = 1.f / L;
        } else {
          // O / (L + 2^(sink - m)), from the larger of the two exponents
          const float sink = a.sink[s.hg * kHG + st] * kLog2e;
          const float M = fmaxf(m, sink);
          if (sink != INFINITY && m != -INFINITY) {
            const float em = exp2f(m - M);
            f = em / (L * em + exp2f(sink - M));
          }
        }
        ms.corr[st] = f;
      }
      soft_bar();
      const bool any = s.c0 < s.c1;
      if (any) role_wait(ms, &ms.pv_done, (chunk - 1) & 1);
      tc_fence_after();
#pragma unroll 1
      for (int sl = 2 * half; sl < 2 * half + 2; ++sl) {
        const int d = sl * 128 + 32 * quad + lane;
        // 32 heads at a time: with 64 the registers spill
        float o[32];
        const auto heads = [&](int hh) {
          if (any) {
            tmem_ld_32x32b_x32(tmem + lane_base + kColO + sl * kHG + hh, o);
            tmem_ld_wait();
          }
          const float4* fac = reinterpret_cast<const float4*>(ms.corr + hh);
#pragma unroll
          for (int g = 0; g < 8; ++g) {
            const float4 f = fac[g];
            o[4 * g] = any ? o[4 * g] * f.x : 0.f;
            o[4 * g + 1] = any ? o[4 * g + 1] * f.y : 0.f;
            o[4 * g + 2] = any ? o[4 * g + 2] * f.z : 0.f;
            o[4 * g + 3] = any ? o[4 * g + 3] * f.w : 0.f;
          }
        };
        if (s.slot >= 0) {
          float big = 0.f;
#pragma unroll 1
          for (int hh = 32; hh >= 0; hh -= 32) {
            heads(hh);
#pragma unroll
            for (int h = 0; h < 32; ++h) big = fmaxf(big, fabsf(o[h]));
          }
          // scaled below 2^15, the scale stored with the dim
          const int e = max(-kExpMax, min(kExpMax, exponent(big) - 14));
          const float f = pow2i(-e);
          part_scale(ta.p, a.ws, s.slot)[d] = pow2i(e);
          uint4* po = part_o(ta.p, a.ws, s.slot) + d;
#pragma unroll 1
          for (int hh = 0; hh < kHG; hh += 32, po += 4 * kDim) {
            if (hh > 0) heads(hh);
#pragma unroll
            for (int g = 0; g < 4; ++g) {
              uint32_t w[4];
#pragma unroll
              for (int i = 0; i < 4; ++i) w[i] = pack_f16(o[8 * g + 2 * i] * f, o[8 * g + 2 * i + 1] * f);
              po[g * kDim] = make_uint4(w[0], w[1], w[2], w[3]);
            }
          }
        } else {
          const int d_rope = kDim - a.out_rope_dims;
          const bool turn = a.out_rope_dims > 0 && d >= d_rope;  // the same for the two lanes of a pair
          float cs = 0.f, sn = 0.f;
          if (turn) {
            cs = ms.cs[1][(d - d_rope) / 2];
            sn = ms.sn[1][(d - d_rope) / 2];
          }
          // lanes 2i and 2i + 1 hold adjacent dims: the even lane stores the
          // pair of one head, the odd lane that of the next
          __nv_bfloat16* out = static_cast<__nv_bfloat16*>(a.O) +
                               ((int64_t)s.bt * a.n_heads + s.hg * kHG + (lane & 1)) * kDim + (d & ~1);
#pragma unroll 1
          for (int hh = 0; hh < kHG; hh += 32, out += 32 * kDim) {
            heads(hh);
#pragma unroll
            for (int h = 0; h < 32; h += 2) {
              const float w = __shfl_xor_sync(0xffffffffu, lane & 1 ? o[h] : o[h + 1], 1);
              float lo = lane & 1 ? w : o[h], hi = lane & 1 ? o[h + 1] : w;
              if (turn) rope_turn(lo, hi, cs, sn);
              *reinterpret_cast<uint32_t*>(out + h * kDim) = pack_bf16(lo, hi);
            }
          }
        }
      }
      tc_fence_before();
      soft_bar();  // the next unit replaces the maxima, factors and sums
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == kSoftWarp0 - 1) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

// Adds the parts of a unit in order ("DeepSeek-V4 内部机制" sink equation):
//   M = max(sink, m_j), O = sum_j 2^{m_j - M} l_j (o_j / l_j) / (sum_j 2^{m_j - M} l_j + 2^{sink - M}).
// A CTA per (eight heads, 512 / G dims, unit), two dims and every G-th part per
// thread.  G = 4 where there are fewer CTAs than SMs otherwise, so that the
// rounds of loads are few: 1 unit of 65 parts takes 7.0 us, 18.8 with G = 1; 64
// units of 2 parts take 5.0 us with G = 1 and 13.7 with G = 4, which forms the
// weights four times.
constexpr int kCombineThreads = 256;
template <int G>
__global__ void __launch_bounds__(kCombineThreads) tree_combine_kernel(const __grid_constant__ TreeArgs ta) {
  const MqaArgs& a = ta.a;
  const TreePlan& p = ta.p;
  constexpr int kPer = kCombineThreads / G;  // threads per group of parts
  __shared__ float W[8][kMaxSplits];
  __shared__ float red[G > 1 ? G - 1 : 1][kPer][17];
  const int groups = a.n_heads / kHG, oct = (int)(blockIdx.x / G) & 7, unit = (int)(blockIdx.x / (8 * G));
  const int bt = groups == 2 ? unit >> 1 : unit, hg = groups == 2 ? unit & 1 : 0, b = bt / a.n_q;
  after_previous();  // the parts are complete
  if (a.n_nodes != nullptr && bt - b * a.n_q >= a.n_nodes[b]) return;
  int first = unit * p.splits, n = p.splits;
  bool second = false;  // parts after the first are first segments of their CTAs: every second slot
  if (p.mode == kTreeEven) {
    const int2 cut = unit_cut(p, a.ws)[unit];
    first = cut.x;
    n = abs(cut.y);
    second = cut.y > 0;
    if (n == 0) return;  // written whole
  }
  const auto slot = [&](int j) -> int64_t { return second && j > 0 ? (first & ~1) + 2 * j : first + j; };
  const int tid = threadIdx.x, g = tid / kPer, d = 2 * (tid % kPer + (int)(blockIdx.x % G) * kPer);
  // the first parts' values are on their way while the weights are formed
  constexpr int kAhead = G > 1 ? 4 : 2;
  uint4 x[kAhead][2];
  float2 sc[kAhead];
  const auto fetch = [&](int j0) {
#pragma unroll
    for (int j = 0; j < kAhead; ++j)
      if (j0 + G * j < n) {
        const uint4* o = part_o(p, a.ws, slot(j0 + G * j)) + oct * kDim + d;
        x[j][0] = __ldcg(o);
        x[j][1] = __ldcg(o + 1);
        sc[j] = __ldcg(reinterpret_cast<const float2*>(part_scale(p, a.ws, slot(j0 + G * j)) + d));
      }
  };
  fetch(g);
  {
    // a warp per head: its weights l_j 2^{m_j - M} over their sum; all of a
    // lane's loads are in flight at once
    const int h = tid >> 5, lane = tid & 31;
    constexpr int kLane = kMaxSplits / 32;
    const float sink = a.sink[hg * kHG + 8 * oct + h] * kLog2e;
    float2 ml[kLane];
#pragma unroll
    for (int i = 0; i < kLane; ++i) {
      ml[i] = make_float2(-INFINITY, 0.f);
      if (lane + 32 * i < n) ml[i] = __ldcg(&part_ml(p, a.ws, slot(lane + 32 * i))[8 * oct + h]);
    }
    float M = sink;
#pragma unroll
    for (int i = 0; i < kLane; ++i) M = fmaxf(M, ml[i].x);
    M = warp_max_f32(M);
    const bool zero = sink == INFINITY || M == -INFINITY;
    float den = 0.f;
#pragma unroll
    for (int i = 0; i < kLane; ++i) {
      if (32 * i >= n) break;
      // in two factors, as l may be 2^124 where m - M is below -126
      const float down = ml[i].x - M;
      float w = !zero && ml[i].x != -INFINITY ? ml[i].y * exp2f(fmaxf(down, -120.f)) * exp2f(fminf(down + 120.f, 0.f)) : 0.f;
      ml[i].y = w;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) w += __shfl_xor_sync(0xffffffffu, w, o);
      den += w;
    }
    if (!zero) den += exp2f(sink - M);
#pragma unroll
    for (int i = 0; i < kLane; ++i)
      if (lane + 32 * i < n) W[h][lane + 32 * i] = zero || ml[i].y == 0.f ? 0.f : ml[i].y / den;
  }
  __syncthreads();
  float acc[8][2];
#pragma unroll
  for (int h = 0; h < 8; ++h) acc[h][0] = acc[h][1] = 0.f;
  for (int j0 = g; j0 < n; j0 += G * kAhead) {
    if (j0 > g) fetch(j0);
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      if (j0 + G * j >= n) break;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const uint32_t w4[4] = {x[j][e].x, x[j][e].y, x[j][e].z, x[j][e].w};
        const float s = e ? sc[j].y : sc[j].x;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          __half2 v;
          memcpy(&v, &w4[i], 4);
          const float2 f = __half22float2(v);
          acc[2 * i][e] = fmaf(W[2 * i][j0 + G * j], f.x * s, acc[2 * i][e]);
          acc[2 * i + 1][e] = fmaf(W[2 * i + 1][j0 + G * j], f.y * s, acc[2 * i + 1][e]);
        }
      }
    }
  }
  if (G > 1) {  // the groups' sums, in order
    if (g > 0) {
#pragma unroll
      for (int i = 0; i < 16; ++i) red[g - 1][tid % kPer][i] = acc[i >> 1][i & 1];
    }
    __syncthreads();
    if (g > 0) return;
#pragma unroll
    for (int k = 0; k < G - 1; ++k)
#pragma unroll
      for (int i = 0; i < 16; ++i) acc[i >> 1][i & 1] += red[k][tid][i];
  }
  const int d_rope = kDim - a.out_rope_dims;
  float cs = 1.f, sn = 0.f;
  const bool turn = a.out_rope_dims > 0 && d >= d_rope;
  if (turn)
    rope_sincos((double)a.q_pos[bt] * -1.0, rope_theta(a.rope_base, (d - d_rope) / 2, a.out_rope_dims), &sn, &cs);
  __nv_bfloat16* out = static_cast<__nv_bfloat16*>(a.O) + ((int64_t)bt * a.n_heads + hg * kHG + 8 * oct) * kDim + d;
#pragma unroll
  for (int h = 0; h < 8; ++h) {
    if (turn) rope_turn(acc[h][0], acc[h][1], cs, sn);
    *reinterpret_cast<uint32_t*>(out + h * kDim) = pack_bf16(acc[h][0], acc[h][1]);
  }
}

int sm_count_tree() {
  static int n = 0;
  if (n == 0) {
    int dev = 0, v = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&v, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || v <= 0) {
      cudaGetLastError();
      return 148;
    }
    n = v;
  }
  return n;
}

TreePlan make_tree_plan(const MqaArgs& a) {
  TreePlan p{};
  const int sms = sm_count_tree();
  p.units = (int64_t)a.batch * a.n_q * (a.n_heads / kHG);
  const int64_t rows = (a.idx ? (int64_t)a.k : a.n_entries) + a.window + a.n_draft;
  const int64_t nch = max64(1, (rows + kRows - 1) / kRows);
  p.splits = 1;
  if (a.splits > 0) {
    p.mode = kTreeFixed;
    p.splits = (int)min64(a.splits, nch);
    p.grid = (int)min64(p.units * p.splits, sms);
    p.slots = p.splits > 1 ? (int)(p.units * p.splits) : 0;
  } else if (p.units >= 8 * sms || (int64_t)a.batch * a.n_q > kMaxNodes || p.units * nch >= (1 << 30)) {
    p.mode = kTreeWhole;
    p.grid = (int)min64(p.units, sms);
  } else {
    p.mode = kTreeEven;
    p.grid = (int)min64(p.units * nch, sms);
    p.slots = 2 * p.grid;
  }
  return p;
}

template <bool FP8>
cudaError_t launch_tree(const CUtensorMap& tmQ, const TreeArgs& t, cudaStream_t s) {
  static unsigned long long asked = 0;
  const cudaError_t e = allow_smem(reinterpret_cast<const void*>(tree_umma_kernel<FP8>), kSmemBytes, &asked);
  if (e != cudaSuccess) return e;
  return forget_smem(launch_overlapped(tree_umma_kernel<FP8>, (unsigned)t.p.grid, kThreads, kSmemBytes, 1, s, tmQ, t),
                     &asked);
}

}  // namespace

// The tensor-core path of csa_tree_mqa (one or two groups of 64 heads).
bool tree_umma_path(const MqaArgs& a) {
  return a.ctx_len != nullptr && a.q_dt == CSA_BF16 && (a.kv_dt == CSA_BF16 || a.kv_dt == CSA_KV_FP8MIX) &&
         a.dim == kDim && a.n_heads % kHG == 0 && a.n_heads <= 2 * kHG &&
         (int64_t)a.batch * a.n_q * a.n_heads < ((int64_t)1 << 28) && a.n_draft <= kMaxDraft &&
         a.q_rope_dims <= kMaxRope && a.out_rope_dims <= kMaxRope;
}

size_t tree_umma_workspace(const MqaArgs& a) {
  const TreePlan p = make_tree_plan(a);
  return p.slots == 0 ? 0 : (size_t)p.slots * kSlotBytes + (p.mode == kTreeEven ? (size_t)p.units * 8 : 0);
}

cudaError_t launch_tree_umma(const MqaArgs& a, cudaStream_t s) {
  TreeArgs t{a, make_tree_plan(a), -1};
  for (int i = 0; a.pages.table != nullptr && i < 31; ++i)
    if (a.pages.page_entries == 1 << i) t.page_shift = i;
  CUtensorMap tmQ;
  if (!make_map_2d(&tmQ, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, a.Q, (uint64_t)a.batch * a.n_q * a.n_heads, kDim, 64,
                   kHG, CU_TENSOR_MAP_SWIZZLE_128B))
    return cudaErrorInvalidValue;
  const cudaError_t e = a.kv_dt == CSA_KV_FP8MIX ? launch_tree<true>(tmQ, t, s) : launch_tree<false>(tmQ, t, s);
  if (e != cudaSuccess || t.p.slots == 0) return e;
  const unsigned octets = (unsigned)(t.p.units * (kHG / 8));
  // G changes the order of the sums, which a fixed split count promises to be
  // the same in any batch: there it follows from that count alone.  (The whole
  // call, G = 1 / 4: 120 units of 2 parts 132 / 147 us, of 16 199 / 205, of 24
  // 253 / 260; one unit of 2 parts 355 / 355, of 16 59.5 / 57.0, of 24 45.8 /
  // 41.9, of 128 49.1 / 27.1.)
  const bool one = t.p.mode == kTreeFixed ? t.p.splits <= kFewParts : octets >= (unsigned)sm_count_tree();
  return one ? launch_overlapped(tree_combine_kernel<1>, octets, kCombineThreads, 0, 1, s, t)
             : launch_overlapped(tree_combine_kernel<4>, 4 * octets, kCombineThreads, 0, 1, s, t);
}

}  // namespace csa
