// Attention of a chunk of new tokens over a paged cache on the tcgen05 tensor cores
// (sm_100a): 64 heads of 512 dims, bf16 queries, bf16 or FP8 pages.
//
// Method: "DeepSeek Technical Reports", sections DSA and CSA; "DeepSeek V4 结构速览",
// sections "CSA（c4a 路线）" and "HCA（c128a 路线）" (selected or all visible entries, then the
// raw sliding window; K = V; a sink per head).
//
// A token's rows are cut into tiles of 128: entry tiles first, then window tiles, so that a
// tile's rows have one format.  Per tile, with rows on the MMA's M and heads on N:
//   S^T[r, h]  = KV[r] . q[h]            (M = 128 rows, N = 64 heads, K = 512)
//   O^T[d, h] += V^T[d, r] P^T[r, h]     (M = 4 x 128 dims, N = 64, K = 128 rows)
// both from the same swizzled shared-memory tile (eight column blocks of 64 dims), so a row
// is read once.  P^T goes through shared memory; S^T and O^T live in TMEM.
//
// What bounds it: the two products of a tile take ~3,200 cycles (at N = 64 an MMA reads 6 KB
// of operands, 48 cycles at 128 bytes a cycle, for 32 cycles of math), and one tile of
// shared memory (128 KB, beside 64 KB of queries) leaves no room for a second: S^T of the next
// tile begins only behind the PV of this one, and the tensor pipe waits another ~2,300 cycles
// for the softmax and the hand-overs.  So the next tile waits in registers: producer warps issue its loads as soon as the current tile is
// stored, they travel under this tile's softmax and PV, and each 128-dim pair is stored the
// moment the PV has read its predecessor; its S^T MMAs start on it.  FP8 rows become bf16 on
// the way to shared memory (code times a power of two: exact).  A whole tile of neighbouring
// bf16 rows, of a page or of new_win, needs no registers: TMA puts each pair in place as soon
// as that is free (windows through registers: a selected FP8 chunk 668 us instead of 618).
// Chosen rows go through registers, since row gathers by TMA (one row of 128 bytes after another)
// moved 9 to 25 bytes a cycle and SM against 55 to 80.  A dense bf16 tile takes 2.8 us (5,500
// cycles), one of chosen bf16 rows 3.7, of FP8 rows 3.9, and a token 8 to 9 us beside its tiles
// (queries, the first tile's maxima, the last PV, the output): 2,048 tokens of 8,176 entries
// 2.69 ms, 4,096 tokens with 512 chosen FP8 rows 622 us.  Measured and not taken: loads
// and softmax in the same warps (10,400 cycles: the softmax's shuffles and shared-memory
// accesses queue behind the loads), and two tiles of 64 rows in turn (M = 64 halves the MMA's
// rate: a dense chunk 27 % slower).
//
// The softmax keeps the maximum lazily (raised only when a tile exceeds it by 2^8, which
// rescales O^T in TMEM) and each thread's sums of its eight heads in registers over the tiles of
// an item: the reduction over the rows runs once per item, so an ordinary tile needs one
// barrier (the OR of "some logit exceeds the maximum") before its probabilities.  Logits, sums,
// O^T and partials are float32; the probabilities alone become bf16 for the PV, since the MMA
// takes both operands in one type and the rows are bf16: half a step, 2^-8 of each weight at
// most (a second MMA for the rest of each weight would double the PV).
//
// CTA: warps 0-7 softmax and output (two per TMEM lane quarter, 32 heads each), warps 8-15
// producers, warp 16 issues every MMA, told by warp 17 when a pair has landed (18-19 idle:
// register shares go by warpgroup).
// Producers walk the CTA's tiles as one stream across its items.
//
// Work item = (token, split of its tiles); CTAs walk the items with stride gridDim.x, the
// longest sequences' first.  Few tokens are split over several CTAs (fp32 partials, combined
// by chunk_merge_kernel), many are not.  The rows' addresses come from a chain of loads
// (selection -> block table -> row), run two tiles ahead of their use.
#include "chunk_common.cuh"
#include "tc_common.cuh"

#include <algorithm>
#include <climits>
#include <utility>

namespace csa {

namespace {

constexpr int kH = 64;            // heads
constexpr int kD = 512;           // head dim = latent dim
constexpr int kHi = 64;           // bf16 dims of an FP8 row
constexpr int kNc = kD - kHi;     // its codes
constexpr int kRows = 128;        // rows per tile
constexpr int kKVBlk = kRows * 128;   // bytes of one column block of the tile
constexpr int kQBlk = kH * 128;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kRescale = 8.0f;      // log2 units
constexpr int kSW = 8;                // softmax warps
constexpr int kPW = 8;                // producer warps, each 16 of a tile's rows
constexpr int kST = 32 * kSW;
constexpr int kBarS = kST + 32;       // threads of a barrier of the softmax and the MMA warp
constexpr int kBarW = 64;             // ... of the watching and the MMA warp
constexpr int kLaunch = 640;
// Registers a thread by warpgroup (2 x softmax, 2 x producers, MMA), out of 5 x 96 at launch.
constexpr int kRegsSoftmax = 80, kRegsProd = 144, kRegsMma = 32;
constexpr int kRegsLaunch = 96;       // 65,536 / 640, whole multiples of 8
// .dec must not raise a warpgroup's count and .inc must not lower it (either faults), and the
// shares must fit what the block was launched with (or .inc waits for good).
static_assert(kRegsSoftmax <= kRegsLaunch && kRegsProd >= kRegsLaunch && kRegsMma <= kRegsLaunch &&
                  2 * kRegsSoftmax + 2 * kRegsProd + kRegsMma <= 5 * kRegsLaunch, "setmaxnreg shares");
constexpr uint32_t kHintNs = 64;
constexpr uint64_t kAfterNs = 100000;  // limit of the waits of a CTA of which one gave up
constexpr uint64_t kDrainNs = 1000000; // what a CTA leaves for its copies and MMAs in flight then
constexpr int kSeqCache = 1024;       // sequences whose boundaries are kept in shared memory
constexpr int kSeqOrder = 64;         // sequences that are taken in order of length
constexpr int kItemList = 1024;       // items of a CTA that are chosen by load
constexpr int kMaxCtas = 160;         // ... of CTAs whose loads a warp keeps in registers
constexpr int kMaxSplit = 32;
constexpr int kNewTag = 1 << 30;      // window rows: new_win's row + kNewTag, or the rings' row

// Tiles of n >= 0 rows (n up to 2^31 - 1).
__host__ __device__ __forceinline__ int tiles_of(int n) { return (int)(((unsigned)n + (kRows - 1)) / kRows); }

struct ChunkTc {
  const __nv_bfloat16 *q, *win, *new_win;
  const int32_t *cu_q, *pos0, *idx, *count;
  const float* sink;
  __nv_bfloat16* out;
  float* lse;
  float *part_o, *part_m, *part_l;   // per item [64][512], [64], [64]
  int* err;
  csa_kv_cache kv;
  int b, N, n_w, m, k, nsplit, items, order, d_rope_out, give_up;
  float scale_log2;
  double inv_freq[kMaxOutRopePairs];
};

// A wait of one of the CTA's roles.  Once one gives up, `failed` (shared memory) says so before
// anything that it should have held back happens, and the outputs from there on are NaN; the
// CTA's later waits stay, with a short limit.
__device__ __forceinline__ void role_wait(uint64_t* bar, uint32_t parity, int* err, volatile int* failed) {
  if (tc::mbar_try_wait_hint(bar, parity, kHintNs)) return;
  const uint64_t t0 = tc::globaltimer();
  while (!tc::mbar_try_wait_hint(bar, parity, kHintNs)) {
    const uint64_t dt = tc::globaltimer() - t0;
    if (dt > kAfterNs && (dt > tc::kWaitLimitNs || *failed)) {
      *failed = 1;
      atomicExch(err, CSA_ERR_TIMEOUT);
      return;
    }
  }
}
// The self-test: the role that acts as if a wait of its own had given up.
enum Role { kSoftmaxRole = 1, kProducerRole = 2, kWatchRole = 3 };
__device__ __forceinline__ void role_start(const ChunkTc& p, int role, volatile int* failed) {
  if (p.give_up == role) {
    *failed = 1;
    atomicExch(p.err, CSA_ERR_TIMEOUT);
  }
}

struct Item {
  int tok, part, seq, i0, p0, t, nsel, ne, w0, tb, te;   // part: tok * nsplit + split
  bool live;
};

// The sequences as the CTAs walk them: boundaries and first positions (in shared memory where
// they fit), and, where the sequences are taken longest first, their order, the boundaries in
// that order and this CTA's items.
struct Seqs {
  // shared memory: cu [kSeqCache + 1], pos0 [kSeqCache], cum [kSeqOrder + 1], ord [kSeqOrder],
  // whether cum and ord hold, the list's length (-1: none), the list
  const int32_t* s;
  static constexpr int kPos0 = kSeqCache + 1, kCum = kPos0 + kSeqCache, kOrd = kCum + kSeqOrder + 1;
  static constexpr int kOrdered = kOrd + kSeqOrder, kListed = kOrdered + 1, kList = kListed + 1;
  static constexpr int kWords = kList + kItemList;
  __device__ __forceinline__ bool ordered() const { return s[kOrdered] != 0; }
  __device__ __forceinline__ const int32_t* cu(const ChunkTc& p) const {
    return p.b <= kSeqCache ? s : p.cu_q;
  }
  __device__ __forceinline__ const int32_t* pos0(const ChunkTc& p) const {
    return p.b <= kSeqCache ? s + kPos0 : p.pos0;
  }
  __device__ __forceinline__ const int32_t* cum(const ChunkTc& p) const {
    return ordered() ? s + kCum : cu(p);
  }
  __device__ __forceinline__ int seq(int j) const { return ordered() ? s[kOrd + j] : j; }
};

// The n-th item of this CTA.  In order of length without a list, every other round runs the
// other way, so that the CTA with the longest items of one round has the shortest of the next.
__device__ __forceinline__ int item_at(const Seqs& q, int n) {
  const int listed = q.s[Seqs::kListed];
  if (listed >= 0) return n < listed ? q.s[Seqs::kList + n] : INT_MAX;
  const int x = q.ordered() && (n & 1) ? gridDim.x - 1 - blockIdx.x : blockIdx.x;
  return n * gridDim.x + x;
}

// Item `item` (whole warp).
__device__ __forceinline__ Item get_item(const ChunkTc& p, const Seqs& q, int item, int lane) {
  Item I;
  const int rank = item / p.nsplit;
  const int split = item - rank * p.nsplit;
  const int32_t* cum = q.cum(p);
  const int j = find_seq(cum, p.b, rank, lane);
  I.live = j < p.b && rank >= cum[0];
  if (!I.live) {
    I.tok = I.part = I.seq = I.i0 = I.p0 = I.t = I.nsel = I.ne = I.w0 = I.tb = I.te = 0;
    return I;
  }
  I.seq = q.seq(j);
  I.i0 = q.cu(p)[I.seq];
  I.tok = I.i0 + (rank - cum[j]);
  I.part = I.tok * p.nsplit + split;
  I.p0 = q.pos0(p)[I.seq];
  I.t = I.p0 + (I.tok - I.i0);
  int ns = 0, nwin = 0;
  I.w0 = 0;
  if (I.t >= 0) {
    ns = p.idx ? min(p.count[I.tok], p.k) : min((I.t + 1) / p.m, p.kv.max_pages * kPageEntries);
    I.w0 = max(0, I.t - p.n_w + 1);
    nwin = I.t - I.w0 + 1;
  }
  I.nsel = max(0, ns);
  I.ne = tiles_of(I.nsel);
  const int tiles = I.ne + tiles_of(nwin);
  I.tb = split * tiles / p.nsplit;
  I.te = (split + 1) * tiles / p.nsplit;
  return I;
}

// This CTA's items, written to `list`: each item, longest sequences first, goes to the CTA
// with the least load so far (whole warp; every CTA finds the same shares).  Neighbouring
// sequences whose items cost about the same are dealt as one group: the least level that
// holds the group's items gives each CTA's number of them, and they are dealt in rounds, so
// that a sequence's early and late tokens spread.  Loads in half tiles; an item costs two
// tiles beside its own (queries, first tile's latency, output).  -1: some CTA's list is full
// (or the shares do not add up): not to be used.
// One token of 44 tiles, 261 of 17 and 666 of 1 to 3: 274 us; dealt by turns 310.
template <class Cost>
__device__ __forceinline__ int share_items(const ChunkTc& p, const int32_t* cum, int32_t* list, int lane,
                                           Cost cost_of) {
  constexpr int Q = kMaxCtas / 32;
  int load[Q], total[Q];                           // of CTA lane + 32 q
#pragma unroll
  for (int q = 0; q < Q; ++q) load[q] = total[q] = 0;
  const int grid = gridDim.x, me = blockIdx.x;
  auto valid = [&](int q) { return lane + 32 * q < grid; };
  int got = 0;
  bool dealt = true;
  for (int j = 0; j < p.b;) {
    const int first = cum[j] * p.nsplit;           // the group: sequences j .. j2 - 1
    const int c0 = cost_of(j);
    float work = 0.f;
    int j2 = j;
    for (; j2 < p.b; ++j2) {
      const int c = cost_of(j2);
      if (4 * c < 3 * c0) break;
      work += (float)(cum[j2 + 1] - cum[j2]) * c;
    }
    const int n = (cum[j2] - cum[j]) * p.nsplit;
    j = j2;
    if (n <= 0) continue;
    const int c = max(4, (int)(work * p.nsplit / n));
    const float rc = 1.f / c;
    // items of this group that a CTA takes below level L
    auto below = [&](int q, int L) {
      return valid(q) && load[q] < L ? (int)((L - 1 - load[q]) * rc) + 1 : 0;
    };
    auto held = [&](int L) {
      int k = 0;
#pragma unroll
      for (int q = 0; q < Q; ++q) k += below(q, L);
      return __reduce_add_sync(0xffffffffu, k);
    };
    long long sum = 0;
    int lo = INT_MAX;
#pragma unroll
    for (int q = 0; q < Q; ++q) {
      sum += load[q];
      if (valid(q)) lo = min(lo, load[q]);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    lo = __reduce_min_sync(0xffffffffu, lo);       // holds none
    int hi = (int)(((long long)n * c + sum) / grid) + c + 2;   // holds them all, rounding or not
    while (hi - lo > 1) {
      const int mid = lo + (hi - lo) / 2;
      if (held(mid) < n) lo = mid; else hi = mid;
    }
    int extra = n - held(lo);                      // of those whose next item lies at the level
    int k[Q];
#pragma unroll
    for (int q = 0; q < Q; ++q) {
      k[q] = below(q, lo);
      const bool more = below(q, hi) > k[q];
      const unsigned b = __ballot_sync(0xffffffffu, more);
      k[q] += more && __popc(b & ((1u << lane) - 1)) < extra ? 1 : 0;
      extra -= __popc(b);                          // (negative: none left)
      load[q] += k[q] * c;
      total[q] += k[q];
    }
    // rounds: all CTAs at first, then those that take more than r items of the group, in order
    int least = INT_MAX;
#pragma unroll
    for (int q = 0; q < Q; ++q) {
      if (valid(q)) least = min(least, k[q]);
    }
    least = __reduce_min_sync(0xffffffffu, least);
    for (int r = lane; r < min(least, kItemList - got); r += 32) list[got + r] = first + r * grid + me;
    got = min(got + least, kItemList);
    int at = first + least * grid;
    for (int r = least;; ++r) {
      int all = 0, before = 0;
      bool mine = false;
#pragma unroll
      for (int q = 0; q < Q; ++q) {
        const unsigned b = __ballot_sync(0xffffffffu, k[q] > r);
        all += __popc(b);
        if (q < me / 32) before += __popc(b);
        if (q == me / 32) {
          before += __popc(b & ((1u << (me % 32)) - 1));
          mine = (b >> (me % 32)) & 1;
        }
      }
      if (!all) break;
      if (mine && got < kItemList) {
        if (lane == 0) list[got] = at + before;
        ++got;
      }
      at += all;
    }
    dealt = dealt && at == first + n;
  }
  int most = 0;
#pragma unroll
  for (int q = 0; q < Q; ++q) most = max(most, total[q]);
  return __reduce_max_sync(0xffffffffu, most) > kItemList || !dealt ? -1 : got;
}

// The tiles of a CTA's items, one after another (empty items skipped).
struct Stream {
  Item it;
  int n, tile;   // item_at(n)
  bool live;
};
__device__ __forceinline__ void stream_settle(Stream& s, const ChunkTc& p, const Seqs& q, int lane) {
  while (s.live && s.tile >= s.it.te) {
    const int item = item_at(q, ++s.n);
    if (item >= p.items) { s.live = false; break; }
    s.it = get_item(p, q, item, lane);
    s.live = s.it.live;
    s.tile = s.it.tb;
  }
}

// One lane's row of a tile, resolved in steps so that no step waits for the one before it:
// the list entry, then the page, then the row's number (-1: no row, zeros).
struct RowRef {
  int e, pg;
  bool window;   // uniform: a window tile (e is already the row's number)
};
__device__ __forceinline__ void row_entry(RowRef& r, const Stream& s, const ChunkTc& p, int row) {
  r.window = false;
  r.e = -1;
  r.pg = -1;
  if (!s.live) return;
  const Item& I = s.it;
  if (s.tile < I.ne) {
    const int pos = s.tile * kRows + row;
    if (pos < I.nsel) r.e = p.idx ? p.idx[(long long)I.tok * p.k + pos] : pos;
  } else {
    r.window = true;
    const int x = (s.tile - I.ne) * kRows + row;
    if (x <= I.t - I.w0) {                         // (past t, w0 + x may pass 2^31)
      const int u = I.w0 + x;
      r.e = u >= I.p0 ? kNewTag + I.i0 + (u - I.p0) : I.seq * p.n_w + u % p.n_w;
    }
  }
}
__device__ __forceinline__ void row_page(RowRef& r, int seq, const ChunkTc& p) {
  if (!r.window && r.e >= 0 && r.e < p.kv.max_pages * kPageEntries)
    r.pg = p.kv.block_table[(long long)seq * p.kv.max_pages + r.e / kPageEntries];
}
__device__ __forceinline__ int row_code(const RowRef& r, const ChunkTc& p) {
  if (r.window) return r.e;
  return (unsigned)r.pg < (unsigned)p.kv.num_pages ? r.pg * kPageEntries + r.e % kPageEntries : -1;
}

// 16 bytes of read-only data that nothing in this CTA reads again.
__device__ __forceinline__ uint4 ldg_stream(const void* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  return v;
}
// What a row that does not exist is read from (a predicate on each load costs more than a
// pointer chosen once per row).
__device__ __align__(128) const uint8_t g_zero_row[kD * 2] = {};
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ void sts16(uint8_t* d, uint32_t a, uint32_t b, uint32_t c, uint32_t e) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};"
               ::"r"(tc::smem_u32(d)), "r"(a), "r"(b), "r"(c), "r"(e) : "memory");
}
__device__ __forceinline__ uint8_t* tile_at(uint8_t* sKV, int row, int cb, int cc) {
  return sKV + cb * kKVBlk + row * 128 + ((cc ^ (row & 7)) << 4);
}

// 16-byte registers a producer thread stages of the next tile, and how many of a plain tile's
// four 128-dim pairs they hold (more in the FP8 kernel, for its window tiles, spilled).
template <bool FP8> constexpr int kStage = FP8 ? 18 : 24;
template <bool FP8> constexpr int kPairs = FP8 ? 2 : 3;

// A producer warp moves 16 rows of the tile; lane = (row of four, 16-byte chunk of eight): rows
// 4 i + lane / 8, i < 4, 128 contiguous bytes of a row at a time (64-byte pieces
// take twice the tag lookups: 1,200 instead of 600 cycles for a tile's 128 loads).  The rows'
// places are shuffled to their lanes ahead of all loads: a shuffle between loads waits behind
// them in the same queue.
//
// bf16 rows: kPairs of a tile's four pairs are staged; the others are loaded into their
// registers as those are stored.

// Numbers of the four rows this lane loads.
__device__ __forceinline__ void row_numbers(int (&c)[4], int code, int lane) {
#pragma unroll
  for (int i = 0; i < 4; ++i) c[i] = __shfl_sync(0xffffffffu, code, 4 * i + (lane >> 3));
}
// Address of a plain row: in the pool, in new_win or in the rings.
__device__ __forceinline__ const char* row_addr(const ChunkTc& p, bool window, int code) {
  const __nv_bfloat16* base = static_cast<const __nv_bfloat16*>(p.kv.rows);
  if (window) base = code >= kNewTag ? p.new_win : p.win;
  const char* a = reinterpret_cast<const char*>(base + (long long)(window ? code & (kNewTag - 1) : code) * kD);
  return code < 0 ? reinterpret_cast<const char*>(g_zero_row) : a;
}
template <int NP, int N>
__device__ __forceinline__ void load_bf16(uint4 (&st)[N], int mb, const ChunkTc& p, bool window,
                                          const int (&c)[4], int lane) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const char* a = row_addr(p, window, c[i]) + 16 * (lane & 7) + 256 * mb;
#pragma unroll
    for (int j = 0; j < 2; ++j) st[8 * (mb % NP) + 2 * i + j] = ldg_stream(a + 128 * j);
  }
}
__device__ __forceinline__ void sts16(uint8_t* d, const uint4& v) { sts16(d, v.x, v.y, v.z, v.w); }
template <int NP, int N>
__device__ __forceinline__ void store_bf16(const uint4 (&st)[N], int mb, uint8_t* sKV, int row0,
                                           int lane) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
#pragma unroll
    for (int j = 0; j < 2; ++j)
      sts16(tile_at(sKV, row0 + 4 * i + (lane >> 3), 2 * mb + j, lane & 7), st[8 * (mb % NP) + 2 * i + j]);
  }
}
// FP8 rows: the whole tile is staged.  Pairs 0-2, a row's 128 codes of a pair being eight lanes'
// chunks: st[4 mb ..+3]; pair 3: the last 64 codes, lane = (row of eight, chunk of four):
// st[12..13], and the 64 bf16 dims: st[14..17].  The scale words of the warp's rows stay with
// their rows' lanes.
__device__ __forceinline__ void load_fp8(uint4 (&st)[kStage<true>], uint2& sc, const int (&c)[4], const ChunkTc& p,
                                         int code, int lane) {
  const uint8_t* rows = static_cast<const uint8_t*>(p.kv.rows);
  const __nv_bfloat16* hi = static_cast<const __nv_bfloat16*>(p.kv.hi);
  int cl[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) cl[i] = __shfl_sync(0xffffffffu, code, 8 * i + (lane >> 2));
  sc = make_uint2(0x7f7f7f7fu, 0x7f7f7f7fu);       // a row that does not exist: zeros times 1
  if (code >= 0)
    sc = __ldg(reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(p.kv.scales) + (long long)code * 8));
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint8_t* a = (c[i] >= 0 ? rows + (long long)c[i] * kNc : g_zero_row) + 16 * (lane & 7);
#pragma unroll
    for (int mb = 0; mb < 3; ++mb) st[4 * mb + i] = ldg_stream(a + 128 * mb);
  }
#pragma unroll
  for (int i = 0; i < 2; ++i)
    st[12 + i] = ldg_stream((cl[i] >= 0 ? rows + (long long)cl[i] * kNc + 384 : g_zero_row) + 16 * (lane & 3));
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint8_t* h = c[i] >= 0 ? reinterpret_cast<const uint8_t*>(hi + (long long)c[i] * kHi) : g_zero_row;
    st[14 + i] = ldg_stream(h + 16 * (lane & 7));
  }
}
// Four codes times 2^k as four bf16 values, exactly.  Fast: two codes to f16 in one conversion,
// one mixed-precision product each (f16 x f16 -> f32, the scale as an f16: `s` holds 2^k in
// both halves), two to a bf16 pair: 222 cycles for a lane's 64 codes, against 329 through
// float conversions and products (and 319 building the bf16 bits with integer operations).
__device__ __forceinline__ uint2 codes_fast(uint32_t w, uint32_t s) {
  uint32_t a, b;
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\t"
      "cvt.rn.f16x2.e4m3x2 %1, h;\n\t}" : "=r"(a), "=r"(b) : "r"(w));
  uint2 o;
#define CSA_PAIR(dst, src)                                                                        \
  asm("{\n\t.reg .b16 l, h, x;\n\t.reg .f32 f, g;\n\tmov.b32 {l, h}, %1;\n\tmov.b32 {x, _}, %2;\n\t" \
      "fma.rn.f32.f16 f, l, x, 0f80000000;\n\tfma.rn.f32.f16 g, h, x, 0f80000000;\n\t"             \
      "cvt.rn.bf16x2.f32 %0, g, f;\n\t}" : "=r"(dst) : "r"(src), "r"(s))
  CSA_PAIR(o.x, a);
  CSA_PAIR(o.y, b);
#undef CSA_PAIR
  return o;
}
// The same for any scale.
__device__ __forceinline__ uint2 codes_slow(uint32_t w, uint32_t scale_byte) {
  float f[4];
  e4m3x4_scaled(w, scale_value(scale_byte), f);
  const __nv_bfloat162 x = __floats2bfloat162_rn(f[0], f[1]), y = __floats2bfloat162_rn(f[2], f[3]);
  return make_uint2(*reinterpret_cast<const uint32_t*>(&x), *reinterpret_cast<const uint32_t*>(&y));
}
// Whether a row's seven scale bytes are all normal f16 powers of two (k in [-14, 15]: maxima of
// a group above 448 * 2^-15 = 0.0137 and up to 1.4e7).  A group of zeros (k = -110) is not: a
// selected chunk of 4,096 tokens takes 1.39 ms with one in every 128th row, 1.80 ms with one in
// every row, and 0.76 ms without (16,384 entries, chosen at random).
__device__ __forceinline__ bool scales_fast(const uint2& sc) {
  bool ok = true;
#pragma unroll
  for (int g = 0; g < 7; ++g) ok &= (((g < 4 ? sc.x : sc.y) >> (8 * (g & 3))) & 0xffu) - 113u <= 142u - 113u;
  return ok;
}
// The lane's chunks of pair mb as bf16, and their store.  Lanes 4-7 of eight store their two
// 16-byte pieces in the other order, so that eight lanes hit 128 distinct bytes.
template <int mb>
__device__ __forceinline__ void convert_fp8(const uint4 (&st)[kStage<true>], const uint2& sc, uint4 (&cv)[8], int lane) {
  const uint32_t word = mb < 2 ? sc.x : sc.y;      // groups 4 (mb / 2) ..+3
  const int shift = mb == 3 ? 16 : 16 * (mb & 1) + 8 * ((lane >> 2) & 1);
#pragma unroll
  for (int x = 0; x < (mb == 3 ? 2 : 4); ++x) {
    const uint4 v = st[4 * mb + x];
    const int row = mb == 3 ? 8 * x + (lane >> 2) : 4 * x + (lane >> 3);
    const uint32_t s = (((__shfl_sync(0xffffffffu, word, row) >> shift) & 0xffu) - 112u) * 0x04000400u;
    const uint2 a = codes_fast(v.x, s), b = codes_fast(v.y, s), c = codes_fast(v.z, s), d = codes_fast(v.w, s);
    cv[2 * x] = make_uint4(a.x, a.y, b.x, b.y);
    cv[2 * x + 1] = make_uint4(c.x, c.y, d.x, d.y);
  }
}
template <int mb>
__device__ __forceinline__ void store_fp8(const uint4 (&st)[kStage<true>], const uint4 (&cv)[8], uint8_t* sKV, int row0,
                                          int lane) {
  const int sw = mb == 3 ? 0 : (lane >> 2) & 1;
#pragma unroll
  for (int x = 0; x < (mb == 3 ? 2 : 4); ++x) {
    const int r = row0 + (mb == 3 ? 8 * x + (lane >> 2) : 4 * x + (lane >> 3));
    const int cb = 2 * mb + sw, cc = 2 * (lane & 3);
    const uint4 u = cv[2 * x], v = cv[2 * x + 1];
    sts16(tile_at(sKV, r, cb, cc + sw), sw ? v : u);
    sts16(tile_at(sKV, r, cb, cc + (sw ^ 1)), sw ? u : v);
  }
  if (mb == 3) {
#pragma unroll
    for (int i = 0; i < 4; ++i) sts16(tile_at(sKV, row0 + 4 * i + (lane >> 3), 7, lane & 7), st[14 + i]);
  }
}
// A warp's part of a pair straight from memory, for a tile with a scale that codes_fast does
// not take: lane = (row of 16, half of the pair's dims), one 16-byte piece after another.
__device__ __forceinline__ void move_fp8_slow(const ChunkTc& p, int code, int mb, uint8_t* sKV, int row, int half) {
  const long long c = code;
#pragma unroll 1
  for (int x = 8 * half; x < 8 * half + 8; ++x) {
    const int d = 128 * mb + 8 * x;
    uint4 v = make_uint4(0u, 0u, 0u, 0u);
    if (code >= 0 && d >= kNc) {
      v = *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p.kv.hi) + c * kHi + (d - kNc));
    } else if (code >= 0) {
      const uint2 w = *reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(p.kv.rows) + c * kNc + d);
      const uint32_t sb = static_cast<const uint8_t*>(p.kv.scales)[c * 8 + d / kScaleGroup];
      const uint2 a = codes_slow(w.x, sb), b = codes_slow(w.y, sb);
      v = make_uint4(a.x, a.y, b.x, b.y);
    }
    sts16(tile_at(sKV, row, 2 * mb + half, x & 7), v);
  }
}

// This warp's part of a pair is in shared memory: publish it (every lane its own writes) and
// arrive once for the warp.
__device__ __forceinline__ void warp_arrive(uint64_t* bar, int lane) {
  tc::fence_proxy_async();
  tc::tc_fence_before();
  __syncwarp();
  if (lane == 0) tc::mbar_arrive(bar);
}

// 32 TMEM lanes x 32 columns, as two pieces of 16 lanes: of piece y, lane l gets TMEM lanes
// 16 y + l / 4 and 8 further, columns 8 g + 2 (l % 4) and the next, as r[y][4 g], r[y][4 g + 1]
// and r[y][4 g + 2], r[y][4 g + 3].  One wait for both.
__device__ __forceinline__ void tmem_ld16x2(uint32_t ta, uint32_t (&r)[2][16]) {
#pragma unroll
  for (int y = 0; y < 2; ++y) {
    uint32_t(&q)[16] = r[y];
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x4.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(q[0]), "=r"(q[1]), "=r"(q[2]), "=r"(q[3]), "=r"(q[4]), "=r"(q[5]), "=r"(q[6]),
          "=r"(q[7]), "=r"(q[8]), "=r"(q[9]), "=r"(q[10]), "=r"(q[11]), "=r"(q[12]), "=r"(q[13]),
          "=r"(q[14]), "=r"(q[15])
        : "r"(ta + ((uint32_t)(16 * y) << 16)) : "memory");
  }
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
  for (int y = 0; y < 2; ++y) {      // no use of a value moves above the wait
#pragma unroll
    for (int i = 0; i < 16; ++i) asm volatile("" : "+r"(r[y][i]) :: "memory");
  }
}

// Four 8 x 8 matrices of 16-bit values, stored transposed: a lane holds row lane / 4, columns
// 2 (lane % 4) and the next, of each; lane 8 i + j gives the address of column j of matrix i.
__device__ __forceinline__ void stmatrix4_trans(uint8_t* d, const uint32_t (&v)[4]) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};"
               ::"r"(tc::smem_u32(d)), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]) : "memory");
}
// 16-byte piece cc of head h's 64-byte row: eight heads' pieces cover all banks.
__device__ __forceinline__ uint8_t* stage_at(uint8_t* stage, int h, int cc) {
  return stage + h * 64 + ((cc ^ ((h >> 1) & 3)) << 4);
}

// A box of the output from shared memory to device memory, by one thread and asynchronously.
__device__ __forceinline__ void tma_store_2d(const CUtensorMap* tm, const void* src, int x, int y) {
  asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%1, %2}], [%3];\n\t"
               "cp.async.bulk.commit_group;"
               ::"l"(tm), "r"(x), "r"(y), "r"(tc::smem_u32(src)) : "memory");
}
// This thread's stores have read shared memory.
__device__ __forceinline__ void tma_store_wait_read() {
  asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
}

// The query heads of a token into shared memory (cp.async, by the producer warps).
__device__ __forceinline__ void load_q(const ChunkTc& p, int tok, uint8_t* sQ, int warp, int lane) {
  const __nv_bfloat16* qb = p.q + (long long)tok * kH * kD;
  for (int h = warp; h < kH; h += kPW) {
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const int c = lane + 32 * x;
      tc::cp_async16(sQ + (c >> 3) * kQBlk + h * 128 + (((c & 7) ^ (h & 7)) << 4), qb + (long long)h * kD + 8 * c, 16);
    }
  }
}

__device__ __forceinline__ float nan_f() { return __int_as_float(0x7fc00000); }

// Weight of rows with reference maximum M (log2 units) and of the sink in a denominator
// taken relative to top = max(M, sink2); neither is NaN when one or both are -inf.
__device__ __forceinline__ float rel_weight(float x, float top) {
  return x == -INFINITY ? 0.f : x == top ? 1.f : exp2f(x - top);
}

template <bool FP8>
__global__ void __launch_bounds__(kLaunch, 1)
    chunk_tc_kernel(const __grid_constant__ CUtensorMap tm_rows,
                    const __grid_constant__ CUtensorMap tm_new,
                    const __grid_constant__ CUtensorMap tm_out, const __grid_constant__ ChunkTc p) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  uint8_t* sKV = base;                            // 8 x 16 KB
  uint8_t* sQ = sKV + 8 * kKVBlk;                 // 8 x 8 KB
  uint8_t* sP = sQ + 8 * kQBlk;                   // 16 KB
  float* s_red = reinterpret_cast<float*>(sP + kRows * 128);   // [4][64]
  float* s_M = s_red + 4 * kH;                    // running reference maximum, log2 units
  float* s_alpha = s_M + kH;
  float* s_sink2 = s_alpha + kH;
  float2* s_rot = reinterpret_cast<float2*>(s_sink2 + kH);   // the output's rotation: sine, cosine
  int* s_flag = reinterpret_cast<int*>(s_rot + kMaxOutRopePairs);
  volatile int* s_failed = s_flag + 1;            // a wait of this CTA gave up
  uint64_t* bar_s = reinterpret_cast<uint64_t*>(s_flag + 4);
  uint64_t* bar_pv = bar_s + 1;                   // [4]
  uint64_t* bar_full = bar_pv + 4;                // [4]: a pair of the tile is in place
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(bar_full + 4);
  uint32_t* s_valid = tmem_holder + 2;            // [4] the tile's rows that exist, a bit each
  uint16_t* s_valid16 = reinterpret_cast<uint16_t*>(s_valid);   // ... as the producers write them
  int32_t* s_cu = reinterpret_cast<int32_t*>(s_valid + 4);   // [Seqs::kWords]
  const Seqs seqs{s_cu};

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  pdl_launch_dependents();
  if (p.b <= kSeqCache) {
    for (int i = tid; i <= p.b; i += kLaunch) s_cu[i] = p.cu_q[i];
    for (int i = tid; i < p.b; i += kLaunch) s_cu[Seqs::kPos0 + i] = p.pos0[i];
  }
  if (tid == 0) {
    s_cu[Seqs::kOrdered] = 0;
    s_cu[Seqs::kListed] = -1;
    *s_failed = 0;
  }
  if (tid < kH) s_sink2[tid] = p.sink[tid] * kLog2e;
  if (tid == 0) {
    tc::mbar_init(bar_s, 1);
    for (int i = 0; i < 4; ++i) tc::mbar_init(bar_pv + i, 1);
    for (int i = 0; i < 4; ++i) tc::mbar_init(bar_full + i, kPW);
    tc::fence_barrier_init();
  }
  if (warp == 0) tc::tmem_alloc(tmem_holder, 512);
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  const uint32_t tmem = *tmem_holder;
  if (p.order && s_cu[p.b] <= p.N) {               // (uniform; b fits the cached part)
    const int32_t* s_pos0 = s_cu + Seqs::kPos0;
    int32_t *s_cum = s_cu + Seqs::kCum, *s_ord = s_cu + Seqs::kOrd;
    // rank of a sequence by the entries its last token sees, longest first
    const int s = tid;
    if (s < p.b) {
      auto rows = [&](int x) {
        const int e = max(0, (s_pos0[x] + (s_cu[x + 1] - s_cu[x])) / p.m);
        return p.idx ? min(e, p.k) : e;
      };
      const int mine = rows(s);
      int r = 0;
      for (int x = 0; x < p.b; ++x) {
        const int other = rows(x);
        r += other > mine || (other == mine && x < s);
      }
      s_ord[r] = s;
    }
    __syncthreads();
    if (tid <= p.b) {
      int c = 0;
      for (int x = 0; x < tid; ++x) c += s_cu[s_ord[x] + 1] - s_cu[s_ord[x]];
      s_cum[tid] = c;
    }
    __syncthreads();
    if (warp == 0) {
      auto cost = [&](int j) {                     // half tiles, the mean of the first and the last token
        const int x = s_ord[j], t0 = s_pos0[x], t1 = t0 + (s_cu[x + 1] - s_cu[x]) - 1;
        auto tiles = [&](int t) {
          const int e = min(max(0, (t + 1) / p.m), p.idx ? p.k : p.kv.max_pages * kPageEntries);
          return tiles_of(e) + tiles_of(min(max(0, t + 1), p.n_w));
        };
        return (tiles(t0) + tiles(t1)) / p.nsplit + 4;
      };
      const int got = share_items(p, s_cum, s_cu + Seqs::kList, lane, cost);
      if (lane == 0) {
        s_cu[Seqs::kListed] = got;
        s_cu[Seqs::kOrdered] = 1;
      }
    }
    __syncthreads();
  }
  const uint32_t tS = tmem, tO = tmem + 64;       // columns [0, 64) S^T; [64, 320) O^T

  if (warp >= kSW + kPW) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsMma));
    // ------------------------------------------------------------------ MMA issuer
    if (warp == kSW + kPW) {
    constexpr uint32_t idS = tc::instr_desc(128, kH, 1, 1, 0, 0);   // K-major x K-major
    constexpr uint32_t idO = tc::instr_desc(128, kH, 1, 1, 1, 1);   // MN-major x MN-major
    const uint64_t dS_a = tc::smem_desc_sw128(tc::smem_u32(sKV), 16, 1024);
    const uint64_t dS_b = tc::smem_desc_sw128(tc::smem_u32(sQ), 16, 1024);
    const uint64_t dO_a = tc::smem_desc_sw128(tc::smem_u32(sKV), kKVBlk, 1024);
    const uint64_t dO_b = tc::smem_desc_sw128(tc::smem_u32(sP), 8192, 1024);
    for (int n = 0, item; (item = item_at(seqs, n)) < p.items; ++n) {
      const Item I = get_item(p, seqs, item, lane);
      if (!I.live) break;
      for (int j = I.tb; j < I.te; ++j) {
#pragma unroll 1
        for (int mb = 0; mb < 4; ++mb) {
          tc::named_bar(4 + mb, kBarW);             // the pair (and, with the first, q) is in place
          tc::tc_fence_after();
          if (tc::elect_one()) {
            const uint64_t a0 = tc::desc_advance(dS_a, 2 * mb * kKVBlk), b0 = tc::desc_advance(dS_b, 2 * mb * kQBlk);
#pragma unroll
            for (int kb = 0; kb < 2; ++kb) {
#pragma unroll
              for (int kk = 0; kk < 4; ++kk)
                tc::mma_f16(tS, tc::desc_advance(a0, kb * kKVBlk + kk * 32),
                            tc::desc_advance(b0, kb * kQBlk + kk * 32), idS, (mb | kb | kk) != 0);
            }
            if (mb == 3) tc::mma_commit(bar_s);
          }
          __syncwarp();
        }
        __syncwarp();
        tc::named_bar(2, kBarS);                    // P^T in place, O^T rescaled
        tc::tc_fence_after();
#pragma unroll 1
        for (int mb = 0; mb < 4; ++mb) {
          if (tc::elect_one()) {
            const uint64_t a0 = tc::desc_advance(dO_a, 2 * mb * kKVBlk);
#pragma unroll
            for (int kk = 0; kk < 8; ++kk)
              tc::mma_f16(tO + mb * kH, tc::desc_advance(a0, kk * 2048), tc::desc_advance(dO_b, kk * 2048), idO,
                          (kk > 0) || (j > I.tb));
            tc::mma_commit(bar_pv + mb);           // column blocks 2 mb, 2 mb + 1 are free
          }
          __syncwarp();
        }
      }
    }
    }
    // A poll of a barrier by the MMA warp itself would wait for the tensor pipe to drain, so a
    // second warp watches the pairs land and hands each over at a named barrier.  (It cannot
    // run ahead: a pair of the next tile lands after this tile's PV has read its place.)
    if (warp == kSW + kPW + 1) {
      role_start(p, kWatchRole, s_failed);
      uint32_t g = 0;
      for (int n = 0, item; (item = item_at(seqs, n)) < p.items; ++n) {
        const Item I = get_item(p, seqs, item, lane);
        if (!I.live) break;
        for (int j = I.tb; j < I.te; ++j, ++g) {
#pragma unroll 1
          for (int mb = 0; mb < 4; ++mb) {
            role_wait(bar_full + mb, g & 1, p.err, s_failed);
            tc::named_bar_arrive(4 + mb, kBarW);
          }
        }
      }
    }
  } else if (warp >= kSW) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsProd));
    // ------------------------------------------------------------------ producers
    const int w = warp - kSW;
    const int row0 = 16 * w;                       // this warp's rows of a tile
    const int myrow = row0 + (lane & 15);          // the one whose place this lane finds out
    role_start(p, kProducerRole, s_failed);
    constexpr int NP = kPairs<FP8>;
    uint4 st[kStage<FP8>];
    uint2 sc = make_uint2(0u, 0u);                 // FP8: the scales of this lane's row, and the
    int c4[4];                                     // numbers of the four rows it loads
    Stream S;
    S.n = 0;
    S.live = item_at(seqs, 0) < p.items;
    S.it.te = S.tile = 0;
    if (S.live) {
      S.it = get_item(p, seqs, item_at(seqs, 0), lane);
      S.live = S.it.live;
      S.tile = S.it.tb;
      stream_settle(S, p, seqs, lane);
    }
    // the first tile's row numbers, loads and queries, then the second tile's rows
    RowRef nx;
    row_entry(nx, S, p, myrow);
    row_page(nx, S.it.seq, p);
    int code = -1;
    bool window = false, whole = false, live = false, new_q = false;
    uint32_t have = 0;                             // rows that exist (twice 16 bits)
    int item = -1;
    auto take = [&]() {   // nx becomes the staged tile; its loads go out; nx is the next one's entries
      live = S.live;
      if (!live) return;
      code = row_code(nx, p);
      window = nx.window;
      new_q = S.n != item;
      item = S.n;
      have = __ballot_sync(0xffffffffu, code >= 0);
      // 128 consecutive bf16 rows that all exist, of one page or of new_win, come by TMA,
      // straight into the tile
      if (window) {
        const int u = S.it.w0 + (S.tile - S.it.ne) * kRows;
        whole = u >= S.it.p0 && u <= S.it.t - (kRows - 1);
      } else {
        whole = !FP8 && !p.idx && S.tile < S.it.nsel / kRows && have == 0xffffffffu;
      }
      row_numbers(c4, code, lane);
      if (FP8 && !window) {
        if constexpr (FP8) load_fp8(st, sc, c4, p, code, lane);
      } else if (!whole) {
#pragma unroll
        for (int mb = 0; mb < NP; ++mb) load_bf16<NP>(st, mb, p, window, c4, lane);
      }
      if (!new_q) {
        ++S.tile;
        stream_settle(S, p, seqs, lane);
        row_entry(nx, S, p, myrow);
      }
    };
    auto queries = [&]() {   // the item's first tile: its queries too
      if (!live || !new_q) return;
      load_q(p, S.it.tok, sQ, w, lane);
      ++S.tile;
      stream_settle(S, p, seqs, lane);
      row_entry(nx, S, p, myrow);
    };
    take();
    queries();
    for (uint32_t n = 0; live; ++n) {
      const bool wait_q = new_q;
      // (the PVs of the tile before end in order, and faster than pairs are stored: a staged tile
      // waits for the first and then for the last)
      auto wait_pv = [&](int mb) {
        if (n > 0) {
          role_wait(bar_pv + mb, (n - 1) & 1, p.err, s_failed);
          tc::tc_fence_after();
        }
      };
      auto ready = [&]() {
        if (lane == 0) s_valid16[w] = (uint16_t)have;
        if (wait_q) tc::cp_async_wait_all();
      };
      if (whole) {
        const CUtensorMap* tm = window ? &tm_new : &tm_rows;
        const int first = window ? code & (kNewTag - 1) : code;   // (lane 0 of warp 0)
#pragma unroll
        for (int mb = 0; mb < 4; ++mb) {
          wait_pv(mb);
          if (mb == 0) ready();
          if (w == 0) {
            tc::fence_proxy_async();
            __syncwarp();
            if (lane == 0) {
              tc::mbar_arrive_expect_tx(bar_full + mb, 2 * kKVBlk);
              tc::tma_load_2d(sKV + 2 * mb * kKVBlk, tm, 128 * mb, first, bar_full + mb);
              tc::tma_load_2d(sKV + (2 * mb + 1) * kKVBlk, tm, 128 * mb + 64, first, bar_full + mb);
            }
          } else {
            warp_arrive(bar_full + mb, lane);
          }
        }
        row_page(nx, S.it.seq, p);
      } else if (FP8 && !window) {
        if constexpr (FP8) {
        if (__all_sync(0xffffffffu, scales_fast(sc))) {
          uint4 cv[8];
          convert_fp8<0>(st, sc, cv, lane);         // while its place is still taken
          wait_pv(0);
          store_fp8<0>(st, cv, sKV, row0, lane);
          ready();
          warp_arrive(bar_full, lane);
          convert_fp8<1>(st, sc, cv, lane);
          wait_pv(3);
          store_fp8<1>(st, cv, sKV, row0, lane);
          warp_arrive(bar_full + 1, lane);
          row_page(nx, S.it.seq, p);
          convert_fp8<2>(st, sc, cv, lane);
          store_fp8<2>(st, cv, sKV, row0, lane);
          warp_arrive(bar_full + 2, lane);
          convert_fp8<3>(st, sc, cv, lane);
          store_fp8<3>(st, cv, sKV, row0, lane);
          warp_arrive(bar_full + 3, lane);
        } else {
          wait_pv(3);
          ready();
          row_page(nx, S.it.seq, p);
#pragma unroll 1
          for (int mb = 0; mb < 4; ++mb) {
            move_fp8_slow(p, code, mb, sKV, myrow, lane >> 4);
            warp_arrive(bar_full + mb, lane);
          }
        }
        }
      } else {
#pragma unroll
        for (int mb = 0; mb < 4; ++mb) {
          if (mb < 2) wait_pv(mb == 0 ? 0 : 3);
          store_bf16<NP>(st, mb, sKV, row0, lane);
          if (mb == 0) ready();
          warp_arrive(bar_full + mb, lane);
          if (mb + NP < 4) load_bf16<NP>(st, mb + NP, p, window, c4, lane);
          if (mb == 2) row_page(nx, S.it.seq, p);
        }
      }
      take();
      if (live && new_q) {
        // the queries in shared memory are read by this tile's S^T for the last time
        role_wait(bar_s, n & 1, p.err, s_failed);
        tc::tc_fence_after();
        queries();
      }
    }
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsSoftmax));
    // ------------------------------------------------------------------ softmax and output
    const int qd = warp & 3, hf = warp >> 2;
    const uint32_t lane_addr = (uint32_t)(qd * 32) << 16;
    const int r0 = 32 * qd + (lane >> 2);          // this thread's rows of S^T: r0 + 8 y, y < 4
    const int h0 = 32 * hf + 2 * (lane & 3);       // ... and heads h0 + 8 g, h0 + 8 g + 1, g < 4
    const int row = qd * 32 + lane;                // its TMEM lane of O^T
    uint32_t ns = 0;                               // tiles so far
    role_start(p, kSoftmaxRole, s_failed);

    for (int n = 0, item; (item = item_at(seqs, n)) < p.items; ++n) {
      const Item I = get_item(p, seqs, item, lane);
      if (!I.live) break;
      bool open = true;                            // some head has no maximum yet: no row, or only -inf
      float lsum[8], ref[8];                       // sums, and reference maxima (log2 units, 0: none)
#pragma unroll
      for (int h = 0; h < 8; ++h) lsum[h] = ref[h] = 0.f;
      for (int j = I.tb; j < I.te; ++j) {
        role_wait(bar_s, ns & 1, p.err, s_failed);
        ++ns;
        tc::tc_fence_after();
        const uint32_t have = s_valid[qd];
        // logits less the reference, log2 units
        // (lg[y]: rows r0 + 16 y, 8 further)
        uint32_t lg[2][16];
        auto logits = [&]() {
          tmem_ld16x2(tS + lane_addr + 32 * hf, lg);
#pragma unroll
          for (int y = 0; y < 2; ++y) {
#pragma unroll
            for (int i = 0; i < 16; ++i)
              lg[y][i] = __float_as_uint(fmaf(__uint_as_float(lg[y][i]), p.scale_log2, -ref[2 * (i >> 2) + (i & 1)]));
          }
          if (have != 0xffffffffu) {
            const uint32_t v = have >> (lane >> 2);
#pragma unroll
            for (int y = 0; y < 2; ++y) {
#pragma unroll
              for (int i = 0; i < 16; ++i)
                if (!((v >> (16 * y + 4 * (i & 2))) & 1u)) lg[y][i] = __float_as_uint(-INFINITY);
            }
          }
        };
        logits();
        // the item's first tile, and any while a head has no maximum, set it
        bool exact = open;
        if (!exact) {
          float top = -INFINITY;
#pragma unroll
          for (int i = 0; i < 32; ++i) top = fmaxf(top, __uint_as_float(lg[i >> 4][i & 15]));
          exact = tc::bar_red_or(3, kST, top > kRescale);
        }
        if (exact) {
          float v[8];
#pragma unroll
          for (int g = 0; g < 4; ++g) {
            v[2 * g] = v[2 * g + 1] = -INFINITY;
#pragma unroll
            for (int y = 0; y < 2; ++y) {
              v[2 * g] = fmaxf(v[2 * g], fmaxf(__uint_as_float(lg[y][4 * g]), __uint_as_float(lg[y][4 * g + 2])));
              v[2 * g + 1] = fmaxf(v[2 * g + 1], fmaxf(__uint_as_float(lg[y][4 * g + 1]), __uint_as_float(lg[y][4 * g + 3])));
            }
          }
#pragma unroll
          for (int o = 4; o < 32; o <<= 1) {
#pragma unroll
            for (int h = 0; h < 8; ++h) v[h] = fmaxf(v[h], __shfl_xor_sync(0xffffffffu, v[h], o));
          }
          if (tid == 0) s_flag[0] = s_flag[2] = 0;   // their last reads are behind a barrier
          if (lane == 0) tma_store_wait_read();    // an item's first P^T comes after this and the barrier
          if (lane < 4) {
#pragma unroll
            for (int g = 0; g < 4; ++g)
              *reinterpret_cast<float2*>(s_red + qd * kH + h0 + 8 * g) = make_float2(v[2 * g], v[2 * g + 1]);
          }
          tc::named_bar(3, kST);
          if (tid < kH) {
            // this tile's maxima, relative to the reference that the logits were taken against
            const float tm = fmaxf(fmaxf(s_red[tid], s_red[kH + tid]), fmaxf(s_red[2 * kH + tid], s_red[3 * kH + tid]));
            float Mn = j > I.tb ? s_M[tid] : -INFINITY, al = 1.f;
            if (Mn == -INFINITY) {                 // its first: the logits were taken against 0
              Mn = tm;
              if (tm == -INFINITY) s_flag[2] = 1;
            } else if (tm > kRescale) {
              Mn += tm;
              al = exp2f(-tm);
              s_flag[0] = 1;
            }
            s_M[tid] = Mn;
            s_alpha[tid] = al;
          }
          tc::named_bar(3, kST);
          if (s_flag[0]) {
#pragma unroll 1
            for (int y = 0; y < 4; ++y) {          // this half's two dim blocks, 32 heads each time
              uint32_t o[32];
              const uint32_t ta = tO + 2 * hf * kH + y * 32 + lane_addr;
              const float* al = s_alpha + 32 * (y & 1);
              tc::tmem_ld32(ta, o);
              tc::tmem_ld_wait(o);
#pragma unroll
              for (int h = 0; h < 32; ++h) {
                o[h] = __float_as_uint(__uint_as_float(o[h]) * al[h]);
                if (h % 8 == 7) asm volatile("" ::: "memory");
              }
              tc::tmem_st32(ta, o);
            }
            tc::tmem_st_wait();
          }
#pragma unroll
          for (int g = 0; g < 4; ++g) {
            const float2 M2 = *reinterpret_cast<const float2*>(s_M + h0 + 8 * g);
            const float2 a2 = *reinterpret_cast<const float2*>(s_alpha + h0 + 8 * g);
            ref[2 * g] = M2.x == -INFINITY ? 0.f : M2.x;   // nothing but -inf gives p = 0, not NaN
            ref[2 * g + 1] = M2.y == -INFINITY ? 0.f : M2.y;
            lsum[2 * g] *= a2.x;
            lsum[2 * g + 1] *= a2.y;
          }
          open = s_flag[2] != 0;
          logits();
          // nobody may overwrite these maxima before everyone has read them
          tc::named_bar(3, kST);
        }
        // probabilities: bf16 into P^T (a row's 128-byte line of 64 heads); the sums take them
        // before that rounding
#pragma unroll
        for (int y = 0; y < 2; ++y) {
#pragma unroll
          for (int g = 0; g < 4; ++g) {
#pragma unroll
            for (int e = 0; e < 4; e += 2) {
              const float p0 = ex2(__uint_as_float(lg[y][4 * g + e])), p1 = ex2(__uint_as_float(lg[y][4 * g + e + 1]));
              lsum[2 * g] += p0;
              lsum[2 * g + 1] += p1;
              const int r = r0 + 16 * y + 4 * e;   // e = 2: the row eight further
              *reinterpret_cast<__nv_bfloat162*>(sP + r * 128 + (((4 * hf + g) ^ (r & 7)) << 4) + 4 * (lane & 3)) =
                  __floats2bfloat162_rn(p0, p1);
            }
          }
        }
        tc::fence_proxy_async();
        tc::tc_fence_before();
        tc::named_bar_arrive(2, kBarS);
      }

      // ---------------------------------------------------------------- the item's output
      if (I.te <= I.tb) {
        if (p.nsplit > 1) {                        // nothing to add: weight 0, O not written
          if (tid < kH) {
            p.part_m[(long long)I.part * kH + tid] = -INFINITY;
            p.part_l[(long long)I.part * kH + tid] = 0.f;
          }
        } else {
          uint4* o = reinterpret_cast<uint4*>(p.out + (long long)I.tok * kH * kD);
          for (int x = tid; x < kH * kD / 8; x += kST) o[x] = make_uint4(0u, 0u, 0u, 0u);
          if (p.lse && tid < kH) p.lse[(long long)I.tok * kH + tid] = s_sink2[tid] * kLn2;
        }
        continue;
      }
#pragma unroll
      for (int o = 4; o < 32; o <<= 1) {
#pragma unroll
        for (int h = 0; h < 8; ++h) lsum[h] += __shfl_xor_sync(0xffffffffu, lsum[h], o);
      }
      tc::named_bar(3, kST);                       // s_red's readers of the last maximum are done
      if (lane < 4) {
#pragma unroll
        for (int g = 0; g < 4; ++g)
          *reinterpret_cast<float2*>(s_red + qd * kH + h0 + 8 * g) = make_float2(lsum[2 * g], lsum[2 * g + 1]);
      }
      tc::named_bar(3, kST);
      if (tid < kH) {
        const float l = s_red[tid] + s_red[kH + tid] + s_red[2 * kH + tid] + s_red[3 * kH + tid];
        const float M = l == 0.f ? -INFINITY : s_M[tid];
        if (p.nsplit > 1) {
          p.part_m[(long long)I.part * kH + tid] = M;
          p.part_l[(long long)I.part * kH + tid] = l;
        } else {
          const float sink2 = s_sink2[tid], top = fmaxf(M, sink2);
          const float wr = rel_weight(M, top);
          const float den = l * wr + rel_weight(sink2, top);
          s_alpha[tid] = den == 0.f ? 0.f : wr / den;
          if (p.lse) p.lse[(long long)I.tok * kH + tid] = den == 0.f ? -INFINITY : (top + log2f(den)) * kLn2;
        }
      } else if (tid < kH + p.d_rope_out / 2 && p.nsplit == 1) {
        float sn, cs;
        rope_angle((double)I.t * p.inv_freq[tid - kH], &sn, &cs);
        s_rot[tid - kH] = make_float2(sn, cs);
      }
      tc::named_bar(3, kST);
      if (p.nsplit > 1) {
        // lanes are neighbouring dims: a head's 32 dims leave as one 128-byte line
#pragma unroll 1
        for (int mb = 0; mb < 4; ++mb) {
          role_wait(bar_pv + mb, (ns - 1) & 1, p.err, s_failed);
          const bool ok = !*s_failed;
          tc::tc_fence_after();
          uint32_t o[32];
          tc::tmem_ld32(tO + mb * kH + 32 * hf + lane_addr, o);
          tc::tmem_ld_wait(o);
          float* dst = p.part_o + ((long long)I.part * kH + 32 * hf) * kD + mb * 128 + row;
#pragma unroll
          for (int h = 0; h < 32; ++h) dst[h * kD] = ok ? __uint_as_float(o[h]) : nan_f();
        }
      } else {
        // A warp's 32 dims of 32 heads of each dim block become [head][dim] rows of 64 bytes in
        // the warp's part of P^T, which the PVs have read by then (stmatrix transposes 8 x 8
        // values at a time), and leave by TMA.  (Pairs exchanged by shuffles and stored in 4
        // bytes queued behind the loads of the producers: a selected chunk 2 % slower, 5 % in bf16.)
        uint8_t* stage = sP + warp * 2048;
        float w[8];
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          const float2 w2 = *reinterpret_cast<const float2*>(s_alpha + h0 + 8 * g);
          w[2 * g] = w2.x;
          w[2 * g + 1] = w2.y;
        }
        const int rope0 = kD - p.d_rope_out;
#pragma unroll 1
        for (int mb = 0; mb < 4; ++mb) {
          role_wait(bar_pv + mb, (ns - 1) & 1, p.err, s_failed);
          tc::tc_fence_after();
          uint32_t ob[2][16];
          tmem_ld16x2(tO + mb * kH + 32 * hf + lane_addr, ob);
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            uint32_t(&o)[16] = ob[y];
            const int d0 = mb * 128 + 32 * qd + 16 * y;   // this lane's dims: d0 + lane / 4, 8 further
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const float f = w[2 * (i >> 2) + (i & 1)];
              o[i] = __float_as_uint(f == 0.f ? 0.f : __uint_as_float(o[i]) * f);
            }
            if (d0 + 16 > rope0) {                        // the other dim of a pair: lane ^ 4
              const int odd = (lane >> 2) & 1;
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                const int u = d0 + 8 * e + (lane >> 2) - rope0;
                const float2 r = u >= 0 ? s_rot[u >> 1] : make_float2(0.f, 1.f);
                const float sn = odd ? -r.x : r.x;
#pragma unroll
                for (int i = 2 * e; i < 16; i += (i & 1) ? 3 : 1) {
                  const float x = __uint_as_float(o[i]);
                  const float z = __shfl_xor_sync(0xffffffffu, x, 4);
                  if (u >= 0) o[i] = __float_as_uint(fmaf(x, r.y, z * sn));
                }
              }
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) {                 // packed in place: o[i] heads 2 i, 2 i + 1
              const __nv_bfloat162 b2 =
                  __floats2bfloat162_rn(__uint_as_float(o[2 * i]), __uint_as_float(o[2 * i + 1]));
              o[i] = *reinterpret_cast<const uint32_t*>(&b2);
            }
          }
          // the stage is free: the last PV has read P^T, the store of the block before its rows
          if (mb == 0) role_wait(bar_pv + 3, (ns - 1) & 1, p.err, s_failed);
          const bool ok = !*s_failed;
          if (lane == 0) tma_store_wait_read();
          __syncwarp();
#pragma unroll
          for (int y = 0; y < 2; ++y) {
#pragma unroll
            for (int a = 0; a < 2; ++a) {                 // 16 heads x 16 dims
              uint32_t v[4];
#pragma unroll
              for (int i = 0; i < 4; ++i) v[i] = ok ? ob[y][4 * a + i] : 0x7fff7fffu;
              const int h = 16 * a + 8 * (lane >> 4) + (lane & 7);
              stmatrix4_trans(stage_at(stage, h, 2 * y + ((lane >> 3) & 1)), v);
            }
          }
          tc::fence_proxy_async();
          __syncwarp();
          if (lane == 0) tma_store_2d(&tm_out, stage, mb * 256 + qd * 64, I.tok * kH + 32 * hf);
        }
      }
      tc::tc_fence_before();
      tc::named_bar(3, kST);                       // s_red, s_alpha and s_M are free again
      if (tid < kH && *s_failed) {
        if (p.nsplit > 1) p.part_l[(long long)I.part * kH + tid] = nan_f();   // the merge's output and lse
        else if (p.lse) p.lse[(long long)I.tok * kH + tid] = nan_f();
      }
    }
    if (lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
  }

  tc::tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    if (*s_failed) {
      const uint64_t t0 = tc::globaltimer();
      while (tc::globaltimer() - t0 < kDrainNs) {}
    }
    tc::tc_fence_after();
    tc::tmem_dealloc(tmem, 512);
  }
}

// Combines the splits of a token: CTA per (token, two heads), four warps a head, four dims a
// thread.  A lane holds one split's weight e^(m_s - top) / den, found by the warp's reductions
// over the splits; the partial rows are added in batches of loads, those of empty splits (not
// written, weight 0) dropped after the load, so that no load waits for another (a branch around
// each took 7.7 us for 8 tokens of 17 splits).
constexpr int kMergeHeads = 2;
__global__ void __launch_bounds__(128 * kMergeHeads) chunk_merge_kernel(const __grid_constant__ ChunkTc p) {
  const int tok = blockIdx.x, lane = threadIdx.x & 31;
  const int h = blockIdx.y * kMergeHeads + (threadIdx.x >> 7), d = 4 * (threadIdx.x & 127);
  const int seq = find_seq(p.cu_q, p.b, tok, lane);
  if (seq >= p.b || tok < p.cu_q[0]) return;
  const int t = p.pos0[seq] + (tok - p.cu_q[seq]);
  const float sink2 = p.sink[h] * kLog2e;
  pdl_wait();
  const long long it0 = (long long)tok * p.nsplit;
  const float m = lane < p.nsplit ? p.part_m[(it0 + lane) * kH + h] : -INFINITY;
  const float l = lane < p.nsplit ? p.part_l[(it0 + lane) * kH + h] : 0.f;
  const float top = fmaxf(warp_max(m), sink2);
  float w = rel_weight(m, top);
  const float den = warp_sum(l * w) + rel_weight(sink2, top);
  w = den == 0.f ? 0.f : w / den;
  if (p.lse && d == 0) p.lse[(long long)tok * kH + h] = den == 0.f ? -INFINITY : (top + log2f(den)) * kLn2;
  float acc[4] = {0.f, 0.f, 0.f, 0.f};
  const float* src = p.part_o + (it0 * kH + h) * kD + d;
#pragma unroll 8
  for (int s = 0; s < p.nsplit; ++s) {
    const float4 v = *reinterpret_cast<const float4*>(src + (long long)s * kH * kD);
    const float ws = __shfl_sync(0xffffffffu, w, s);
    acc[0] = ws == 0.f ? acc[0] : fmaf(v.x, ws, acc[0]);
    acc[1] = ws == 0.f ? acc[1] : fmaf(v.y, ws, acc[1]);
    acc[2] = ws == 0.f ? acc[2] : fmaf(v.z, ws, acc[2]);
    acc[3] = ws == 0.f ? acc[3] : fmaf(v.w, ws, acc[3]);
  }
#pragma unroll
  for (int u = 0; u < 4; u += 2) {
    const int x = d + u - (kD - p.d_rope_out);
    if (x >= 0 && p.d_rope_out > 0) {
      float sn, cs;
      rope_angle((double)t * p.inv_freq[x >> 1], &sn, &cs);
      const float y0 = fmaf(acc[u], cs, acc[u + 1] * sn), y1 = fmaf(acc[u + 1], cs, -acc[u] * sn);
      acc[u] = y0; acc[u + 1] = y1;
    }
  }
  const __nv_bfloat162 lo = __floats2bfloat162_rn(acc[0], acc[1]), hi = __floats2bfloat162_rn(acc[2], acc[3]);
  uint2 v;
  v.x = *reinterpret_cast<const uint32_t*>(&lo);
  v.y = *reinterpret_cast<const uint32_t*>(&hi);
  *reinterpret_cast<uint2*>(p.out + ((long long)tok * kH + h) * kD + d) = v;
}

constexpr size_t kSmem = 1024 + 8 * kKVBlk + 8 * kQBlk + kRows * 128 + (4 * kH + 3 * kH) * 4 + kMaxOutRopePairs * 8 + 16 + 9 * 8 + 8 + 16 +
                         Seqs::kWords * 4;
static_assert(kSmem <= 227 * 1024, "shared memory per CTA");

thread_local int t_give_up = 0;   // csa_selftest_chunk_give_up: of this thread's next call

int sm_count() {
  int dev = 0, sms = 148;
  cudaGetDevice(&dev);
  cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  return sms;
}

// Splits per token.  In units of a tile's time: a CTA's item of n tiles costs about n + 1.5 (its
// queries, the first tile's latency, the output), the CTAs work through ceil(N splits / SMs)
// items each, and the partials of an item about 0.015 in all.  With two tokens per SM or more
// splitting only multiplies the items' overhead (and their tokens may be far shorter than
// L_max says): never.
int splits_for(int tiles, int N, int sms) {
  int best = 1;
  double least = 0;
  if (N >= 2 * sms) return best;
  for (int ns = 1; ns <= std::min(kMaxSplit, std::max(tiles, 1)); ++ns) {
    const double rounds = (double)(((long long)N * ns + sms - 1) / sms);
    const double cost = rounds * ((tiles + ns - 1) / ns + 1.5) + (ns > 1 ? 1.0 + 0.015 * N * ns : 0.0);
    if (ns == 1 || cost < least) { best = ns; least = cost; }
  }
  return best;
}
// Tiles of a token with L visible positions.
int token_tiles(int n_w, int m, int k, int L) {
  return tiles_of(k > 0 ? k : L / m) + tiles_of(std::max(n_w, 0));
}
int plan_splits(int n_w, int m, int k, int N, int L_max) {
  return splits_for(token_tiles(n_w, m, k, L_max), N, sm_count());
}

// Most items with partials among the calls of up to N tokens and L_max positions.  Every tile
// count from the first position's to the last's occurs; over kPlanTiles of them (and then they
// are not tried one by one) all splits may be taken.
constexpr int kPlanTiles = 4096;
long long plan_items_bound(int n_w, int m, int k, int N, int L_max) {
  const int sms = sm_count(), top = std::min(N, 2 * sms - 1);
  const int first = token_tiles(n_w, m, k, 1), last = token_tiles(n_w, m, k, L_max);
  if (last > kPlanTiles) return (long long)top * kMaxSplit;
  long long most = 0;
  for (int tiles = last; tiles >= first; --tiles) {
    for (int n = top; n > 0 && (long long)n * std::min(kMaxSplit, tiles) > most; --n) {
      const int ns = splits_for(tiles, n, sms);
      if (ns > 1) most = std::max(most, (long long)n * ns);
    }
  }
  return most;
}

}  // namespace

bool chunk_tc_supported(int H, int d, int dtype, int d_rope_out, const csa_kv_cache& kv) {
  if (H != kH || d != kD || dtype != CSA_BF16 || d_rope_out > 2 * kMaxOutRopePairs) return false;
  if ((long long)kv.num_pages * kPageEntries > INT_MAX) return false;
  return kv.dtype == CSA_BF16 || (kv.dtype == CSA_FP8_E4M3 && kv.d_hi == kHi);
}

int chunk_tc_launch_count(int n_w, int m, int k, int N, int L_max) {
  return plan_splits(n_w, m, k, N, L_max) > 1 ? 2 : 1;
}

size_t chunk_tc_workspace_bytes(int n_w, int m, int k, int N, int L_max) {
  const int ns = plan_splits(n_w, m, k, N, L_max);
  return ns > 1 ? (size_t)N * ns * kH * (kD + 2) * 4 : 0;
}

size_t chunk_tc_workspace_bound(int n_w, int m, int k, int N, int L_max) {
  return (size_t)plan_items_bound(n_w, m, k, N, L_max) * kH * (kD + 2) * 4;
}

bool chunk_tc_give_up(int role) {
  if (role < kSoftmaxRole || role > kWatchRole) return false;
  t_give_up = role;
  return true;
}

csa_status launch_chunk_attn_tc(const ChunkArgs& a, const csa_kv_cache& kv, void* ws,
                                size_t ws_bytes, cudaStream_t st) {
  // row numbers of the window and of q carry a tag in bit 30
  if ((long long)a.b * a.n_w >= kNewTag || a.N >= kNewTag) return CSA_ERR_UNSUPPORTED;
  ChunkTc p{};
  p.q = static_cast<const __nv_bfloat16*>(a.q);
  p.win = static_cast<const __nv_bfloat16*>(a.win);
  p.new_win = static_cast<const __nv_bfloat16*>(a.new_win);
  p.cu_q = a.cu_q; p.pos0 = a.pos0; p.idx = a.idx; p.count = a.count; p.sink = a.sink;
  p.out = static_cast<__nv_bfloat16*>(a.out); p.lse = a.lse; p.kv = kv;
  p.b = a.b; p.N = a.N; p.n_w = a.n_w; p.m = a.m; p.k = a.k; p.d_rope_out = a.d_rope_out;
  p.give_up = std::exchange(t_give_up, 0);
  p.scale_log2 = a.scale * kLog2e;
  p.err = device_error_word();
  if (!p.err) return CSA_ERR_CUDA;
  rope_frequencies(p.inv_freq, a.d_rope_out, a.theta);
  p.nsplit = plan_splits(a.n_w, a.m, a.k, a.N, a.L_max);
  const long long items = (long long)a.N * p.nsplit;
  if (items > INT_MAX - (1 << 20)) return CSA_ERR_UNSUPPORTED;   // a round past the last fits too
  p.items = (int)items;
  if (p.nsplit > 1) {
    if (!ws || ws_bytes < (size_t)items * kH * (kD + 2) * 4 || (reinterpret_cast<uintptr_t>(ws) & 15))
      return CSA_ERR_INVALID_ARG;
    p.part_o = static_cast<float*>(ws);
    p.part_m = p.part_o + items * kH * kD;
    p.part_l = p.part_m + items * kH;
  }
  auto kern = kv.dtype == CSA_FP8_E4M3 ? chunk_tc_kernel<true> : chunk_tc_kernel<false>;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmem) != cudaSuccess)
    return CSA_ERR_CUDA;
  // bf16 pages as one matrix of rows, copied in column blocks of 64 dims of a tile's 128 rows
  CUtensorMap tm{};
  if (kv.dtype == CSA_BF16 &&
      !make_tmap_2d_b16(&tm, kv.rows, kD, (uint64_t)kv.num_pages * kPageEntries, 64, kRows))
    return CSA_ERR_CUDA;
  CUtensorMap tm_new{};
  if (a.n_w >= kRows && a.N >= kRows &&            // (a whole tile of new rows needs both)
      !make_tmap_2d_b16(&tm_new, a.new_win, kD, (uint64_t)a.N, 64, kRows))
    return CSA_ERR_CUDA;
  // the output as rows of one head, stored in boxes of 32 dims of 32 heads
  CUtensorMap tm_out{};
  if (p.nsplit == 1 && !make_tmap_2d_u8_swz(&tm_out, a.out, kD * 2, (uint64_t)a.N * kH, 64, 32, 64))
    return CSA_ERR_CUDA;
  const int grid = (int)std::min<long long>(items, sm_count());
  // Several rounds of items of several sequences: longest first, each to the CTA with the least
  // load.  (One token of 44 tiles before 927 of 1 to 17: 434 us in the given order, 274 so; more
  // sequences than kSeqOrder even out by themselves, and sorting them would take long.)
  p.order = p.items > grid && a.b > 1 && a.b <= kSeqOrder && grid <= kMaxCtas;
  if (csa_launch(kern, dim3(grid), dim3(kLaunch), kSmem, st, false, tm, tm_new, tm_out, p) != cudaSuccess) return CSA_ERR_CUDA;
  if (p.nsplit > 1 &&
      csa_launch(chunk_merge_kernel, dim3(a.N, kH / kMergeHeads), dim3(128 * kMergeHeads), 0, st, true, p) != cudaSuccess)
    return CSA_ERR_CUDA;
  return CSA_OK;
}

}  // namespace csa
