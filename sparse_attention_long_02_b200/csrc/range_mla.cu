// range_mla.cu -- MLA attention over ranges of the latent cache, sm_100a: every
// earlier key (dense), or a sliding window and the first few keys (sinks).
//
// Row t of a contiguous cache sits at position p = q_pos0 + t; query j of
// sequence b of a paged cache at p = seq_len[b] - nq + j. It sees the keys s
// with s <= min(p, last key) and, with a window w, s > p - w or s < sinks:
//   out = sum_s exp(z_s - lse) kv[s, :512],  z_s = sm_scale q . kv[s],
//   lse = log sum_s exp(z_s).
// A row that sees no key gets out = 0 and lse = -inf. What a row does not see has
// no effect on it; an infinite value that it does see with no weight (logit -inf)
// makes that dim NaN, any other infinity or NaN the whole row.
//
// Row tiles. The MMA's M holds 128 rows: all heads of G = min(queries, 128 / H)
// consecutive queries of one sequence, which share the keys they read. A row
// tile's keys are 64-key units (cache blocks) that any of its queries sees,
// the sinks' units first, then the window's; two units form a tile of 128 keys.
//
// Two roles in a cluster of two CTAs. A 128 x 512 fp32 output fills the 512
// TMEM columns of an SM, so one SM cannot hold it beside the logits. CTA 0
// forms the logits and the softmax, CTA 1 the output:
//   CTA 0: Q's 512 latent dims move into TMEM (256 columns; the rope dims stay
//     in shared memory), K's latent dims stream through a ring of TMA loads (128
//     keys x 128 dims an entry), its rope dims through a place of their own;
//     S = Q K^T (M = 128, N = 128, K = 576) goes into one of two TMEM buffers; two
//     groups of four warps (thread = row) take 64 keys of a tile each: row
//     maximum, running reference maximum (re-based only when it grows by more
//     than 8 in log2 units), P = exp2(z - m) in bf16 into shared memory, one 16 KB
//     bulk copy per 64 keys into CTA 1.
//   CTA 1: V chunks (64 keys x 256 dims) stream through their own ring;
//     O (+)= P V (M = 128, N = 256 twice, K = 64); eight warps rescale O in
//     TMEM when a reference maximum moved, and write the result.
// Nothing below fp32 crosses but P, which the PV product takes in bf16: half a step
// (2^-8) of each weight at most, which for many keys averages out below the
// output's own rounding (error of the outputs against 64 bits 1.7e-3 to 1.8e-3,
// 1.5e-3 to 1.7e-3 with P in fp32). l sums P before that rounding.
//
// Each role streams its own operand, K from HBM and V, the same rows two tiles
// later, from L2. (Asking L2 for tiles ahead of the loads does not pay: its lines
// are lost again before they are used; 64 x 32768 tokens read 797 MB for 456 when
// it ran six tiles ahead.)
//
// Work split. The tiles of all row tiles form one list; each cluster takes an
// equal share of it, wherever it begins and ends (or whole row tiles in turn,
// where that is as fast as equal shares and the join they need). A row tile
// inside one share is written directly; one cut over several clusters leaves its
// parts (fp32 sums of p v with the row's maximum and sum) in the workspace, which
// range_join_kernel combines: with m = max m_i, l = sum l_i 2^(m_i - m),
// O = sum O_i 2^(m_i - m) / l.
//
// What bounds it. A tile's MMAs take CTA 0 2400 cycles and CTA 1 2050, and CTA
// 0's shared memory takes 368 KB a tile in and out (K in and to the MMA, the rope
// dims of Q, P in and out), 2900 cycles at 128 B each. Measured, a tile takes 3400
// cycles with the cache in L2 (64 sequences of 32768 tokens that share 37 MB: 472
// us), where the softmax's 2700 and its waits set the pace and QK waits 450 for a
// buffer, and 3850 from HBM (20 calls in a row 595 us, 4.1 TB/s), where QK waits
// 1000 for K. Those are held at 1.5 GHz of 1.97 by the board's 1000 W, and a loop of
// calls that lasts seconds at 1.37 GHz (692 us, 3.5 TB/s). Short calls run at full
// clock, and their time is the way to the first tile (9 us), the shares' tiles (2 to
// 2.3 us each), a part's way to memory (5 us: an SM writes some 30 B a cycle) and
// the join (7 us): one sequence of 131072 tokens 62 us.
//
// CTA 0's shared memory is full to the last bytes. The rope dims of K in a place of
// their own, not in the ring, took 64 x 32768 from 635 to 595 us; what paid for
// them are the barriers of CTA 1 alone, which live in its own memory, and one
// buffer of maxima instead of two. Paying with a staging of P instead makes the
// softmax wait for its copies (three stagings: 580 us with the cache in L2, where
// it was 508; one a unit and five ring entries: 707), and entries of 16 KB cost a
// wait and a commit more each (598 us).
#include <algorithm>
#include <cstddef>

#include "common.cuh"
#include "dsa_internal.h"
#include "split.cuh"

namespace dsa {
namespace {

constexpr int kThreads = 512;
constexpr int kAtom = 128 * 128;                // 128 rows (or keys) x 64 dims, 128-B swizzled
constexpr int kUnitAtom = 64 * 128;             // 64 keys x 64 dims
constexpr int kEntry = 2 * kAtom;               // ring entry: 128 dims of 128 rows
constexpr int kVChunk = 4 * kUnitAtom;          // 64 keys x 256 dims
// Even, so that each of the two loading warps has its own places and sees every
// phase of their barriers.
constexpr int kRing = 4;
constexpr int kQPairs = 4;                      // Q dims [0, 512) live in TMEM, 128 at a time
constexpr uint32_t kColQ = 256;                 // after two buffers of 128 logits
constexpr int kPieces = 8;                      // pieces written down at a time
constexpr int kPSlots = 4;
constexpr int kVRing = 4;
constexpr float kRebase = 8.0f;                 // lazy rescale threshold (log2 units)
constexpr int kMaxClusters = 74;                // of two CTAs, one on each of 148 SMs
constexpr int kScanItems = 16384;               // row tiles a cluster scans for its share
constexpr int kItemCost = 3;                    // a row tile's fixed cost, in tiles
// What cutting row tiles costs, in tiles: where there are fewer of them than
// clusters a cluster writes one part, else two. (Two queries of 64 sequences in a
// window of 2048: 94 to 116 us whole, 117 to 131 us cut; a prompt of 8191 rows and a
// window of 1024: 2.74 ms whole, 2.76 ms cut; 64 x 32768 tokens: 638 us whole, 626 us
// cut; one sequence of 131072: 2004 us whole, 61 us cut. In turn on one board.)
constexpr int kCutCostFew = 5, kCutCostMany = 7;
// Tiles whose sums the tensor core adds up before they move to a second sum in
// memory. Its fp32 additions cut where they do not round, so a sum of n keys of
// like weights comes out too small by up to n / 16 2^-23: measured 0.02% at 32768
// keys, 0.08% at 131072, 0.6% at a million (more than the output's rounding), 10%
// at 16 million.
constexpr int kSumTiles = 1024;

struct LogitsSmem {                             // CTA 0
  uint8_t ring[kRing][kEntry];                  // K's latent dims, and Q on its way to TMEM
  uint8_t k_rope[kAtom];                        // K dims [512, 576)
  uint8_t p[2][2][kAtom];                       // staging of P, by tile parity and unit
  uint8_t q_rope[kAtom];                        // Q dims [512, 576)
  float alpha[2][128];                          // staging of the rescale factors, by tile parity
  float mx[2][128];                             // a tile's maxima, by softmax group
};
struct OutputSmem {                             // CTA 1
  uint8_t p[kPSlots][kAtom];
  uint8_t v[kVRing][kVChunk];
  float alpha[4][128];                          // rescale factors, by tile
  float2 ml[2][128];                            // reference maximum and sum of each softmax group
  uint8_t stage[8][32 * 64];                    // output rows on their way out, by warp
  unsigned lost[128][16];                       // by row, a bit a dim: see clean_v
  unsigned long long v_full[kVRing], v_empty[kVRing];
  unsigned long long p_full[kPSlots], p_free[kPSlots];
  unsigned long long al_full[4];                // a tile's rescale factors have landed
  unsigned long long o_ok[4];                   // O is ready for a tile's PV
  unsigned long long clean[2];                  // V of a tile's unit with hidden keys is ready
  unsigned long long pv_done[4];
  unsigned long long ml_full;
  unsigned long long piece_done[kPieces];       // the piece's output is on its way
};
constexpr size_t kBig = std::max(sizeof(LogitsSmem), sizeof(OutputSmem));
static_assert(kBig % 1024 == 0, "the control block follows the larger role's memory");
// Scratch of the search for the share. It may still run in CTA 1 when CTA 0's
// first atoms of P arrive (the cluster's barrier is passed on arrival, before the
// search), so it lies where no copy or load lands in either CTA: CTA 1's staging
// of output rows, and at the same place in CTA 0 a staging of P, which only that
// CTA's softmax writes, after the search.
constexpr size_t kScratch = offsetof(OutputSmem, stage);
constexpr size_t kScratchBytes = 2 * (kThreads / 32) * sizeof(long long);
static_assert(kScratchBytes <= sizeof(OutputSmem::stage) && kScratch % 8 == 0 &&
                  kScratch >= offsetof(LogitsSmem, p) &&
                  kScratch + kScratchBytes <= offsetof(LogitsSmem, q_rope),
              "the search's scratch is out of reach of copies and loads");

// The bits a .. b of 0 .. 63 (none if a > b).
__device__ __forceinline__ unsigned long long range_bits(int a, int b) {
  a = max(a, 0);
  b = min(b, 63);
  if (a > b) return 0ull;
  return (~0ull >> (63 - b)) & (~0ull << a);
}

// A row tile: its rows, positions and 64-key units.
struct Item {
  long long row0;                               // first row of q, out and lse
  int nrows;
  int pos0, posl;                               // positions of its first and last query
  int last;                                     // last key of the sequence
  int ns, w0, nu;                               // units: 0 .. ns-1, then w0 on; nu in all
  int tiles;                                    // of two units, at least one
  const int* table;                             // the sequence's block table (paged)
};

// (Out of line: the search for the share, which calls it first, has then
// fetched its code for the warp that walks the pieces.)
__device__ __noinline__ Item item_geom(const RangeArgs& A, int i) {
  Item x;
  int nq;
  if (A.block_table) {
    const int b = i / A.per_seq, j0 = (i - b * A.per_seq) * A.G;
    nq = min(A.G, A.nq - j0);
    const int len = max(0, min(A.seq_len[b], A.max_blocks * 64));
    x.pos0 = len - A.nq + j0;
    x.last = len - 1;
    x.row0 = (static_cast<long long>(b) * A.nq + j0) * A.H;
    x.table = A.block_table + static_cast<long long>(b) * A.max_blocks;
  } else {
    const int j0 = i * A.G;
    nq = min(A.G, A.T - j0);
    x.pos0 = A.q_pos0 + j0;
    x.last = A.S - 1;
    x.row0 = static_cast<long long>(j0) * A.H;
    x.table = nullptr;
  }
  x.nrows = nq * A.H;
  x.posl = x.pos0 + nq - 1;
  const int hi = min(x.posl, x.last);
  const int lo = A.window ? max(0, x.pos0 - A.window + 1) : 0;
  int w1 = 0;
  x.ns = x.w0 = 0;
  if (hi >= 0) {
    if (lo <= hi) {
      x.w0 = lo >> 6;
      w1 = (hi >> 6) + 1;
    }
    if (A.window && A.sinks) {
      x.ns = (min(A.sinks, hi + 1) + 63) >> 6;
      if (w1 == 0) {
        x.w0 = w1 = x.ns;
      } else if (x.ns >= x.w0) {
        x.ns = x.w0 = 0;
      }
    }
  }
  x.nu = x.ns + w1 - x.w0;
  x.tiles = max(1, (x.nu + 1) >> 1);
  return x;
}

__device__ __forceinline__ int unit_block(const Item& x, int u) {
  return u < x.ns ? u : x.w0 + u - x.ns;
}
__device__ __forceinline__ int tile_units(const Item& x, int t) {
  return x.nu - 2 * t >= 2 ? 2 : 1;
}
// The keys of unit u (bits) that some query of the row tile does not see, though
// they are loaded: past the first query's position, or before the last query's
// window (and no sink).
__device__ __forceinline__ unsigned long long unit_hidden(const RangeArgs& A, const Item& x, int u) {
  const int kb = unit_block(x, u) * 64;
  unsigned long long hidden = range_bits(min(x.pos0, x.last) + 1 - kb, 63);
  if (A.window) hidden |= range_bits(A.sinks - kb, x.posl - A.window - kb);
  return hidden;
}
// Cache row of unit u's first key, or kv_rows (whose loads give zeros) when
// the row tile has no keys or the block id is out of range. In two steps, so
// that a tile's table entries can be on their way while the tile before is
// loaded.
__device__ __forceinline__ int unit_entry(const RangeArgs& A, const Item& x, int u) {
  if (u >= x.nu) return -1;
  const int block = unit_block(x, u);
  return A.block_table ? __ldg(x.table + block) : block;
}
__device__ __forceinline__ int entry_row(const RangeArgs& A, int entry) {
  const bool bad = entry < 0 || (A.block_table && entry >= A.nblk);
  return bad ? A.kv_rows : entry * 64;
}

// A cluster's share, one piece (tiles [t0, t1) of a row tile) after another.
struct Piece {
  Item x;
  long long start;                              // the row tile's place in the weight list
  int item;                                     // -1: no more pieces
  int t0, t1;
  bool first, last;                             // holds the row tile's first, last tile
};
static_assert(sizeof(Piece) % 4 == 0 && sizeof(Piece) <= 128, "at most a word a lane");

struct Walk {
  int item, off, whole;
  long long left, start;
  __device__ __forceinline__ explicit Walk(const Share& s)
      : item(s.item), off(s.off), whole(s.whole), left(s.left), start(s.start) {}
  __device__ __forceinline__ Piece next(const RangeArgs& A) {
    Piece p;
    p.item = -1;
    if (whole) {
      // later rows of a prefill see more keys: they go first
      if (item < A.items) {
        p.item = A.items - 1 - item;
        item += A.clusters;
        p.x = item_geom(A, p.item);
        p.t0 = 0;
        p.t1 = p.x.tiles;
        p.first = p.last = true;
      }
      return p;
    }
    while (left > 0 && item < A.items) {
      p.x = item_geom(A, item);
      const int weight = p.x.tiles + kItemCost;
      const int take = static_cast<int>(min(static_cast<long long>(weight - off), left));
      p.t0 = max(0, off - kItemCost);
      p.t1 = off + take - kItemCost;
      p.start = start;
      p.first = p.t0 == 0;
      p.last = p.t1 == p.x.tiles;
      left -= take;
      off = 0;
      start += weight;
      ++item;
      if (p.t1 > p.t0) {
        p.item = item - 1;
        break;
      }
    }
    return p;
  }
};

struct Ctl {
  Piece piece[kPieces];                         // by piece number
  // CTA 0
  unsigned long long q_free;                    // the piece's last QK is done
  unsigned long long q_ready[kQPairs];          // 128 dims of Q are in TMEM
  unsigned long long rope_full;
  unsigned long long k_full[kRing], k_empty[kRing];
  unsigned long long kr_full, kr_empty;         // k_rope
  unsigned long long s_full[2], s_empty[2];     // by tile parity
  unsigned long long mx_bar[4];                 // both groups' maxima of a lane quarter
  // by tile parity and unit, so that whoever waits on one sees every phase
  unsigned long long p_own[2][2];               // a staged atom is written
  unsigned long long p_ack[2][2];               // CTA 1 holds the atom: its staging is free
  unsigned long long p_room[kPSlots];           // CTA 1 has room for another atom
  unsigned long long ml_free;                   // CTA 1 has read ml
  unsigned long long o_done;                    // CTA 1's PV of a piece; the give-up path
  Share share;                                  // of the row tiles' weights
  unsigned long long piece_full[kPieces];
  uint32_t tmem_base;
  int abort_flag[2];                            // and the CTA's progress: tiles of QK, of PV
};
constexpr size_t kSmemBytes = kBig + sizeof(Ctl);
static_assert(kSmemBytes <= 232448, "fits the 227 KB of shared memory a CTA may use");

__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{\n\t.reg .b64 a, b, c, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
      "mov.b64 c, {%6, %7};\n\tfma.rn.f32x2 d, a, b, c;\n\tmov.b64 {%0, %1}, d;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 a, b, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
      "add.rn.f32x2 d, a, b;\n\tmov.b64 {%0, %1}, d;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}

// The sign bits of a word's two bf16 that are NaN or infinite.
__device__ __forceinline__ unsigned not_finite(uint32_t w) {
  return ((w & 0x7f807f80u) + 0x00800080u) & 0x80008000u;
}
// This thread's 16-byte pieces of a V chunk's rows k0 .. k1 - 1: piece i is of row
// k0 + i / 4, in atom i % 4 (rows of 128 B, 16-B chunk c of row k at c ^ (k % 8)).
constexpr int kCleaners = 256;                  // threads
__device__ __forceinline__ uint4* v_piece(uint8_t* v, int k0, int i, int sub) {
  return reinterpret_cast<uint4*>(v + (i & 3) * kUnitAtom + (k0 + (i >> 2)) * 128 + (sub & 7) * 16);
}
// Turns the NaN and infinite values of those pieces into 0.
//
// An infinite value v of a key that a row sees with logit -inf makes p v = 0 inf, a
// NaN, of that dim of the row; with any other logit the whole row is NaN. So the
// dims are noted in `lost` for the rows that see the key. `key0` is the key of the
// chunk's row 0, `dim0` its first dim.
__device__ __noinline__ void clean_v(const RangeArgs& A, uint8_t* v, int k0, int k1, int sub, int key0,
                                     int dim0, int pos0, int last, int nrows, unsigned (*lost)[16],
                                     unsigned long long& o_ok, uint32_t parity,
                                     volatile int* abort_flag, unsigned* err) {
  bool ready = false;
#pragma unroll 1
  for (int i = sub >> 3; i < 4 * (k1 - k0); i += kCleaners / 8) {
    uint32_t* w = reinterpret_cast<uint32_t*>(v_piece(v, k0, i, sub));
    unsigned dims = 0;                          // of the piece's eight
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const unsigned bad = not_finite(w[e]);
      if (!bad) continue;
      if (bad & 0x8000u) w[e] &= 0xffff0000u;
      if (bad >> 31) w[e] &= 0x0000ffffu;
      dims |= ((bad >> 15 & 1u) | (bad >> 30 & 2u)) << (2 * e);
    }
    if (!dims) continue;
    const int k = k0 + (i >> 2), s = key0 + k;
    const int dim = dim0 + 64 * (i & 3) + 8 * ((sub ^ k) & 7);
#pragma unroll 1
    for (int r = 0; r < nrows; ++r) {
      const int pos = pos0 + r / A.H;
      if (s > min(pos, last) || (A.window && s <= pos - A.window && s >= A.sinks)) continue;
      // once all warps have come to this tile, none has to read what the piece
      // before has lost
      if (!ready && !wait1(o_ok, parity, abort_flag, err)) return;
      ready = true;
      atomicOr(&lost[r][dim >> 5], dims << (dim & 31));
    }
  }
}
// Adds the 256 dims of O (of each lane's row) to the sum in memory, scaled for the
// reference maximum of now (`fresh`: there is none yet), and starts O anew; at a
// piece's `end` adds that sum to O instead. Each thread meets its own floats only.
__device__ __noinline__ void move_sum(float4* sum, int pitch, bool valid, float scale, bool fresh,
                                      bool end, uint32_t o_cols) {
#pragma unroll 1
  for (int cc = 0; cc < 8; ++cc) {
    float o[32];
    tmem_ld32(o_cols + 32 * cc, o);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      float4* at = sum + static_cast<long long>(8 * cc + e) * pitch;
      float4 a = make_float4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
      if (valid && !fresh) {
        const float4 old = *at;
        a = make_float4(fmaf(old.x, scale, a.x), fmaf(old.y, scale, a.y), fmaf(old.z, scale, a.z),
                        fmaf(old.w, scale, a.w));
      }
      if (valid && !end) *at = a;
      o[4 * e] = end ? a.x : 0.f;
      o[4 * e + 1] = end ? a.y : 0.f;
      o[4 * e + 2] = end ? a.z : 0.f;
      o[4 * e + 3] = end ? a.w : 0.f;
    }
    tmem_st32(o_cols + 32 * cc, o);
  }
}
// Makes the noted dims (256 from TMEM column o_cols on) of each lane's row NaN, and
// forgets them.
__device__ __noinline__ void spoil_lost(unsigned* lost, uint32_t o_cols) {
#pragma unroll 1
  for (int cc = 0; cc < 8; ++cc) {
    const unsigned bits = lost[cc];
    lost[cc] = 0;
    float o[32];
    tmem_ld32(o_cols + 32 * cc, o);
#pragma unroll
    for (int e = 0; e < 32; ++e)
      if ((bits >> e) & 1u) o[e] = __int_as_float(0x7fffffff);
    tmem_st32(o_cols + 32 * cc, o);
  }
}

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
range_mla_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                 const __grid_constant__ CUtensorMap tm_v,
                 const __grid_constant__ RangeArgs A) {
  extern __shared__ __align__(1024) uint8_t big[];              // (swizzled tiles start on 1024 B)
  LogitsSmem& sl = *reinterpret_cast<LogitsSmem*>(big);
  OutputSmem& so = *reinterpret_cast<OutputSmem*>(big);
  Ctl& ctl = *reinterpret_cast<Ctl*>(big + kBig);
  unsigned* err = A.err;
  const uint32_t rank = cluster_rank(), peer = rank ^ 1u;
  const int cluster = static_cast<int>(blockIdx.x >> 1);
  const int warp = warp_id(), lane = lane_id();

  // The barriers and the tensor memory are made ready while the share is found;
  // the other CTA's are known to be by the end of that.
  if (warp == 15) {
    auto init = [](unsigned long long& b, int count) { mbar_init(smem_u32(&b), count); };
    const int i = lane & 7;
    if (lane < 4) {
      init(ctl.q_ready[i], 4);
      init(ctl.k_full[i], 1);
      init(ctl.k_empty[i], 1);
      init(ctl.mx_bar[i], 2);
      init(ctl.p_own[i >> 1][i & 1], 4);
      init(ctl.p_ack[i >> 1][i & 1], 1);
      init(ctl.p_room[i], 1);
      if (rank == 1) {
        init(so.v_full[i], 1);
        init(so.v_empty[i], 1);
        init(so.p_full[i], 1);
        init(so.p_free[i], 1);
        init(so.al_full[i], 1);
        init(so.o_ok[i], 8);
        init(so.pv_done[i], 1);
        // CTA 1 expects the first atoms of P before CTA 0 can send one
        mbar_expect_tx(smem_u32(&so.p_full[i]), kAtom);
        mbar_expect_tx(smem_u32(&so.al_full[i]), 512);
      }
    } else if (lane >= 8 && lane < 16) {
      init(ctl.piece_full[i], 1);
      if (rank == 1) init(so.piece_done[i], 1);
    } else if (lane == 16 || lane == 17) {
      init(ctl.s_full[i], 1);
      init(ctl.s_empty[i], 8);
      if (rank == 1) init(so.clean[i], 8);
    } else if (lane == 18) {
      init(ctl.q_free, 1);
      init(ctl.rope_full, 1);
      init(ctl.kr_full, 1);
      init(ctl.kr_empty, 1);
      init(ctl.ml_free, 8);
      init(ctl.o_done, 1);
      if (rank == 1) init(so.ml_full, 8);
      ctl.abort_flag[0] = launch_aborted(err) ? 1 : 0;
      ctl.abort_flag[1] = 0;
    }
    fence_barrier_init();
  } else if (warp == 1) {
    tmem_alloc(smem_u32(&ctl.tmem_base), 512);
    tmem_relinquish();
  }
  __syncwarp();
  cluster_arrive();
  if (A.whole) {
    if (threadIdx.x == 0) {
      ctl.share = Share{};
      ctl.share.item = cluster;
      ctl.share.whole = 1;
    }
  } else {
    find_share<kThreads>(ctl.share, reinterpret_cast<long long*>(big + kScratch), A.items, cluster,
                         A.clusters, A.items < A.clusters ? kCutCostFew : kCutCostMany,
                         [&](int i) {
                           if (A.block_table && blockIdx.x == 0) {
                             const int len = A.seq_len[i / A.per_seq];
                             if (len < 0 || len > A.max_blocks * 64) raise_error(err, kErrBounds);
                           }
                           return item_geom(A, i).tiles + kItemCost;
                         });
  }
  static_assert(sizeof(so.lost) == kThreads * sizeof(uint4), "one store a thread");
  if (rank == 1) reinterpret_cast<uint4*>(so.lost)[threadIdx.x] = make_uint4(0, 0, 0, 0);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  // each CTA works out the first piece for itself
  Walk walk(ctl.share);
  Piece p;
  if (warp == 13) {
    p = walk.next(A);
    if (lane == 0) {
      ctl.piece[0] = p;
      mbar_arrive(smem_u32(&ctl.piece_full[0]));
    }
    __syncwarp();
  }
  cluster_wait();
  const uint32_t tmem = ctl.tmem_base;
  volatile int* abort_flag = ctl.abort_flag;
  bool ok = *abort_flag == 0;
  // The later pieces are written down by CTA 1's warp 13 for every role of both
  // CTAs (the arithmetic is cold code that each role would wait for between two
  // pieces).
  Item& x = p.x;
  int pieces = 0;                               // of this role so far
  auto next_piece = [&](bool whole_warp) {
    unsigned long long& full = ctl.piece_full[pieces & (kPieces - 1)];
    const uint32_t parity = (pieces / kPieces) & 1;
    ok = ok && (whole_warp ? wait32<true>(full, parity, abort_flag, err)
                           : wait1<true>(full, parity, abort_flag, err));
    if (!ok) return false;
    p = ctl.piece[pieces & (kPieces - 1)];
    return p.item >= 0;
  };

  if (rank == 0) {
    if (warp == 0 || warp == 2) {
      // ------------------------------------------------ Q and K loads (CTA 0)
      // Two warps take the ring's entries in turn: a wait, an expect and four
      // loads cost one thread about 540 cycles (1200 while the TMA unit is busy
      // with others), an entry's MMAs 549. In a piece's first tile each K entry
      // follows the Q entry it meets. The first warp then loads Q's rope dims,
      // the second those of each tile of K.
      const int par = warp >> 1;
      if (lane == 0) {
        int ent = 0, loaded = 0, ropes = 0;
        for (; next_piece(false); ++pieces) {
          const int q_row = static_cast<int>(x.row0);
          int e0 = unit_entry(A, x, 2 * p.t0), e1 = unit_entry(A, x, 2 * p.t0 + 1);
          for (int t = p.t0; ok && t < p.t1; ++t) {
            const int n = tile_units(x, t);
            const int c0 = entry_row(A, e0), c1 = entry_row(A, e1);
            e0 = unit_entry(A, x, 2 * t + 2);
            e1 = unit_entry(A, x, 2 * t + 3);
            const bool with_q = t == p.t0;
            const int count = with_q ? 2 * kQPairs : kQPairs;
#pragma unroll 1
            for (int i = par; i < count; i += 2) {
              const int at = ent + i, st = at & (kRing - 1);
              if (at >= kRing &&
                  !(ok = wait1(ctl.k_empty[st], (at / kRing + 1) & 1, abort_flag, err)))
                break;
              loaded = at + 1;
              const uint32_t full = smem_u32(&ctl.k_full[st]), dst = smem_u32(sl.ring[st]);
              const int ch = 2 * (with_q ? i >> 1 : i);           // first 64-dim chunk
              mbar_expect_tx(full, with_q && par == 0 ? kEntry : 2 * n * kUnitAtom);
              if (with_q && par == 0) {
                tma_load_2d(dst, &tm_q, full, 64 * ch, q_row);
                tma_load_2d(dst + kAtom, &tm_q, full, 64 * ch + 64, q_row);
              } else {
                tma_load_3d(dst, &tm_k, full, 0, c0, ch);
                if (n > 1) tma_load_3d(dst + kUnitAtom, &tm_k, full, 0, c1, ch);
                tma_load_3d(dst + kAtom, &tm_k, full, 0, c0, ch + 1);
                if (n > 1) tma_load_3d(dst + kAtom + kUnitAtom, &tm_k, full, 0, c1, ch + 1);
              }
            }
            if (!ok) break;
            ent += count;
            if (par == 0 && with_q) {
              // the rope dims of Q, once the piece before no longer reads its own
              if (pieces > 0 && !(ok = wait1(ctl.q_free, (pieces - 1) & 1, abort_flag, err))) break;
              mbar_expect_tx(smem_u32(&ctl.rope_full), kAtom);
              tma_load_2d(smem_u32(sl.q_rope), &tm_q, smem_u32(&ctl.rope_full), 512, q_row);
              ++ropes;
            } else if (par == 1) {
              // and of K
              if (ropes > 0 && !(ok = wait1(ctl.kr_empty, (ropes - 1) & 1, abort_flag, err))) break;
              const uint32_t full = smem_u32(&ctl.kr_full), dst = smem_u32(sl.k_rope);
              mbar_expect_tx(full, n * kUnitAtom);
              tma_load_3d(dst, &tm_k, full, 0, c0, 2 * kQPairs);
              if (n > 1) tma_load_3d(dst + kUnitAtom, &tm_k, full, 0, c1, 2 * kQPairs);
              ++ropes;
            }
          }
        }
        if (!ok) {           // let the loads in flight land before this CTA leaves
          for (int c = max(0, loaded - kRing); c < loaded; ++c)
            if ((c & 1) == par)
              mbar_drain(smem_u32(&ctl.k_full[c & (kRing - 1)]), (c / kRing) & 1);
          if (ropes > 0)
            mbar_drain(smem_u32(par == 0 ? &ctl.rope_full : &ctl.kr_full), (ropes - 1) & 1);
        }
      }
    } else if (warp >= 12) {
      // ------------------------------------------- Q into TMEM (CTA 0)
      // Row r of each entry, bf16 pairs, lane = row; once the piece before no
      // longer reads Q. (That wait also means every entry of that piece has
      // been consumed, so the barriers waited on below are in the phase before.)
      const int r = 32 * (warp & 3) + lane;
      const uint32_t q_cols = tmem + (static_cast<uint32_t>(32 * (warp & 3)) << 16) + kColQ;
      int ent = 0;
      for (; next_piece(true); ++pieces) {
        if (pieces > 0 && !(ok = wait32(ctl.q_free, (pieces - 1) & 1, abort_flag, err))) break;
        tc_fence_after();
#pragma unroll 1
        for (int j = 0; j < kQPairs; ++j) {
          const int e = ent + 2 * j, st = e & (kRing - 1);
          if (!(ok = wait32(ctl.k_full[st], (e / kRing) & 1, abort_flag, err))) break;
#pragma unroll
          for (int half = 0; half < 4; ++half) {
            const uint4* row =
                reinterpret_cast<const uint4*>(sl.ring[st] + (half >> 1) * kAtom + r * 128);
            uint32_t pk[16];
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              const uint4 v = row[(4 * (half & 1) + c) ^ (r & 7)];
              pk[4 * c] = v.x;
              pk[4 * c + 1] = v.y;
              pk[4 * c + 2] = v.z;
              pk[4 * c + 3] = v.w;
            }
            tmem_st16(q_cols + 64 * j + 16 * half, pk);
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(&ctl.q_ready[j]));
        }
        ent += kQPairs * (p.t1 - p.t0 + 1);
      }
    } else if (warp == 1) {
      // ------------------------------------------------------- QK (CTA 0)
      // One thread. The barriers of the next entry and of the next tile's
      // buffer are asked for before the MMAs ahead of them are issued, so that
      // a satisfied wait costs nothing after them.
      if (elect_one()) {
        const uint32_t id2 = idesc_bf16(128, 128, false), id1 = idesc_bf16(128, 64, false);
        const uint64_t ring_d = sdesc_sw128(smem_u32(sl.ring[0]), 0, 1024);
        const uint64_t rope_d = sdesc_sw128(smem_u32(sl.q_rope), 0, 1024);
        const uint64_t kr_d = sdesc_sw128(smem_u32(sl.k_rope), 0, 1024);
        const uint32_t k_full = smem_u32(&ctl.k_full[0]), k_empty = smem_u32(&ctl.k_empty[0]);
        int ent = 0, tc = 0;
        auto ask = [&](int e) {
          return mbar_try_wait(k_full + 8 * (e & (kRing - 1)), (e / kRing) & 1);
        };
        auto full = [&](int e, bool there) {
          return there || wait1(ctl.k_full[e & (kRing - 1)], (e / kRing) & 1, abort_flag, err);
        };
        // debug: ml_free completes only after an output is written, so this
        // bounded wait runs out and both CTAs leave through their give-up paths
        if (ok && (debug_bits(err) & kDbgStallMla)) ok = wait1(ctl.ml_free, 0, abort_flag, err);
        bool room = true;                               // the tile's buffer of logits is free
        for (; next_piece(false); ++pieces) {
          for (int t = p.t0; ok && t < p.t1; ++t, ++tc) {
            const int sb = tc & 1;
            const uint32_t d = tmem + 128 * sb;
            const uint32_t id = tile_units(x, t) > 1 ? id2 : id1;
            const bool first = t == p.t0;
            bool there = !first && ask(ent);
            if (!room && !(ok = wait1(ctl.s_empty[sb], ((tc >> 1) + 1) & 1, abort_flag, err)))
              break;
            tc_fence_after();
#pragma unroll 1
            for (int j = 0; j < kQPairs; ++j, ++ent) {
              if (first) {                              // Q has left its place in the ring
                if (!(ok = wait1(ctl.q_ready[j], pieces & 1, abort_flag, err))) break;
                mbar_arrive(k_empty + 8 * (ent & (kRing - 1)));
                ++ent;
                tc_fence_after();
              }
              if (!(ok = full(ent, there))) break;
              there = !first && j + 1 < kQPairs && ask(ent + 1);
              const int st = ent & (kRing - 1);
              const uint64_t kd = ring_d + st * (kEntry >> 4);
              const uint32_t qc = tmem + kColQ + 64 * j;
#pragma unroll
              for (int kk = 0; kk < 8; ++kk)            // 16 dims: 8 TMEM columns of Q
                mma_bf16_ts(d, qc + 8 * kk, kd + (kk >> 2) * (kAtom >> 4) + 2 * (kk & 3), id,
                            (j > 0 || kk > 0) ? 1u : 0u);
              mma_commit(k_empty + 8 * st);
            }
            if (!ok) break;
            if (first && !(ok = wait1(ctl.rope_full, pieces & 1, abort_flag, err))) break;
            if (!(ok = wait1(ctl.kr_full, tc & 1, abort_flag, err))) break;
            room = tc == 0 || mbar_try_wait(smem_u32(&ctl.s_empty[sb ^ 1]),
                                            (((tc + 1) >> 1) + 1) & 1);
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) mma_bf16(d, rope_d + 2 * kk, kr_d + 2 * kk, id, 1u);
            mma_commit(smem_u32(&ctl.kr_empty));
            mma_commit(smem_u32(&ctl.s_full[sb]));
            abort_flag[1] = tc;
            if (t + 1 == p.t1) mma_commit(smem_u32(&ctl.q_free));
          }
        }
        if (!ok) {           // MMAs in flight read shared memory: wait for them
          mma_commit(smem_u32(&ctl.o_done));
          mbar_drain(smem_u32(&ctl.o_done), 0);
        }
      }
      __syncwarp();
    } else if (warp == 3) {
      // ----------------------------------------------- P to CTA 1 (CTA 0)
      if (lane == 0) {
        int a = 0, tc = 0;
        unsigned sent = 0;                              // parity of each staging's count
        for (; next_piece(false); ++pieces) {
          for (int t = p.t0; ok && t < p.t1; ++t, ++tc) {
            const int g = tc & 1, n = tile_units(x, t);
#pragma unroll 1
            for (int u = 0; u < n; ++u, ++a) {
              const int slot = a & 3, bit = 2 * g + u;
              if (!(ok = wait1(ctl.p_own[g][u], (sent >> bit) & 1, abort_flag, err))) break;
              if (a >= kPSlots &&
                  !(ok = wait1<true>(ctl.p_room[slot], ((a >> 2) + 1) & 1, abort_flag, err)))
                break;
              // The rescale factors go into tile tc - 4's place: p_room says
              // that PV of the atom four before is done, which is that tile's
              // or a later one's, and PV waits for its tile's rescale.
              if (u == 0)
                bulk_copy_to_peer(mapa(smem_u32(so.alpha[tc & 3]), peer), smem_u32(sl.alpha[g]),
                                  512, mapa(smem_u32(&so.al_full[tc & 3]), peer));
              bulk_copy_to_peer(mapa(smem_u32(so.p[slot]), peer), smem_u32(sl.p[g][u]), kAtom,
                                mapa(smem_u32(&so.p_full[slot]), peer));
              sent ^= 1u << bit;
            }
          }
        }
        // a copy reads this CTA's staging until it lands (a staging never
        // used is in the phase that its parity names as done)
        for (int b = 0; b < 4; ++b) {
          const uint32_t bar = smem_u32(&ctl.p_ack[b >> 1][b & 1]), parity = ((sent >> b) & 1) ^ 1;
          if (!mbar_wait<true>(bar, parity, abort_flag, err)) mbar_drain(bar, parity);
        }
      }
    } else {
      // -------------------------------------------------- softmax (CTA 0)
      // Thread = row; group g takes unit g of every tile. P is formed at once
      // with the reference maximum of the tile before, while the tile's own
      // maximum is found; the two groups then swap maxima, and only where the
      // reference has to move is P formed again. (A piece's first tile looks
      // for its maximum first.)
      const int g = (warp - 4) >> 2;
      const int wq = warp & 3;                          // TMEM lane quarter
      const int r = 32 * wq + lane;                     // row = TMEM lane
      const uint32_t lanes = static_cast<uint32_t>(32 * wq) << 16;
      const float2 scale2 = make_float2(A.sm_scale_log2, A.sm_scale_log2);
      int tc = 0;
      unsigned acked = 3u;                              // parity of each staging's uses, before the first
      for (; next_piece(true); ++pieces) {
        const int pos = x.pos0 + r / A.H;
        const int hi = r < x.nrows ? min(pos, x.last) : -1;
        const int lo = A.window ? pos - A.window + 1 : 0;
        const int sink_hi = A.window ? min(A.sinks - 1, hi) : -1;
        float m = -INFINITY, l = 0.f;
        for (int t = p.t0; ok && t < p.t1; ++t, ++tc) {
          const int n = tile_units(x, t), b = tc & 1, un = 2 * t + g;
          unsigned long long see = 0ull;                // keys of the unit that the row sees
          if (un < x.nu) {
            const int block = unit_block(x, un);
            bool good = true;
            if (A.block_table) {
              const int pb = __ldg(x.table + block);
              good = pb >= 0 && pb < A.nblk;
              if (!good && lane == 0) raise_error(err, kErrBounds);
            }
            const int kb = block * 64;
            if (good) see = range_bits(lo - kb, hi - kb) | range_bits(0, sink_hi - kb);
          }
          const uint32_t s_cols = tmem + lanes + 128 * b + 64 * g;
          const bool first = t == p.t0;
          // the staging is free once CTA 1 holds what it held (a barrier not
          // yet used passes for the phase before its first)
          if (g < n) {
            if (!(ok = wait32<true>(ctl.p_ack[b][g], (acked >> b) & 1, abort_flag, err))) break;
            acked ^= 1u << b;
          }
          if (!(ok = wait32(ctl.s_full[b], (tc >> 1) & 1, abort_flag, err))) break;
          tc_fence_after();
          uint8_t* row = sl.p[b][g] + r * 128;
          float mx = -INFINITY, alpha = 1.f;
          float2 sum2 = make_float2(0.f, 0.f);
#pragma unroll 1
          for (int round = 0; round < 2; ++round) {
            // P = exp2(z - m) of the unit into the staging (not in the first
            // tile's first round), its sum, and the unit's maximum
            const bool form = !first || round == 1;
            const float base = m == -INFINITY ? 0.f : m;
            const float2 base2 = make_float2(-base, -base);
            sum2 = make_float2(0.f, 0.f);
#pragma unroll 1
            for (int h = 0; h < 2 && g < n; ++h) {
              float s[32];
              tmem_ld32(s_cols + 32 * h, s);
              const unsigned bits = static_cast<unsigned>(see >> (32 * h));
              if (!__all_sync(0xffffffffu, bits == ~0u)) {
#pragma unroll
                for (int e = 0; e < 32; ++e)
                  if (!((bits >> e) & 1u)) s[e] = -INFINITY;
              }
              float pm[4] = {mx, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
              for (int e = 0; e < 32; ++e) pm[e & 3] = fmaxf(pm[e & 3], s[e]);
              mx = fmaxf(fmaxf(pm[0], pm[1]), fmaxf(pm[2], pm[3]));
              if (!form) continue;
              // row r of the atom: 128 B, 16-B chunk c at chunk c ^ (r % 8)
#pragma unroll
              for (int c = 0; c < 4; ++c) {
                uint32_t pk[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                  float2 v =
                      fma2(make_float2(s[8 * c + 2 * e], s[8 * c + 2 * e + 1]), scale2, base2);
                  v.x = fast_exp2(v.x);
                  v.y = fast_exp2(v.y);
                  sum2 = add2(sum2, v);
                  const __nv_bfloat162 pb = __floats2bfloat162_rn(v.x, v.y);
                  pk[e] = *reinterpret_cast<const uint32_t*>(&pb);
                }
                *reinterpret_cast<uint4*>(row + (((4 * h + c) ^ (r & 7)) << 4)) =
                    make_uint4(pk[0], pk[1], pk[2], pk[3]);
              }
            }
            if (round == 1) break;
            // the row's maximum over both units; the other group has read the
            // tile before's once it is done with its logits
            if (tc > 0 && !(ok = wait32(ctl.s_empty[b ^ 1], ((tc - 1) >> 1) & 1, abort_flag, err)))
              break;
            sl.mx[g][r] = mx;
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&ctl.mx_bar[wq]));
            if (!(ok = wait32(ctl.mx_bar[wq], tc & 1, abort_flag, err))) break;
            const float top = fmaxf(mx, sl.mx[g ^ 1][r]) * A.sm_scale_log2;
            const float m_new = top > m + kRebase ? top : m;
            const bool moved = m_new != m;
            if (moved && m > -INFINITY) alpha = fast_exp2(m - m_new);
            m = m_new;
            if (!first && !__any_sync(0xffffffffu, moved)) break;
          }
          if (!ok) break;
          if (g == 0) sl.alpha[b][r] = alpha;
          l = l * alpha + (sum2.x + sum2.y);
          fence_proxy_async_smem();                     // generic writes -> bulk-copy reads
          tc_fence_before();
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(smem_u32(&ctl.s_empty[b]));     // the buffer is free for another tile
            if (g < n) mbar_arrive(smem_u32(&ctl.p_own[b][g]));
          }
        }
        if (!ok) break;
        // the group's maximum and sum go to CTA 1
        if (pieces > 0 && !(ok = wait32<true>(ctl.ml_free, (pieces - 1) & 1, abort_flag, err)))
          break;
        const uint32_t ml = mapa(smem_u32(&so.ml[g][r]), peer);
        st_cluster_f32(ml, m);
        st_cluster_f32(ml + 4, l);
        __syncwarp();
        if (lane == 0) mbar_arrive_remote(mapa(smem_u32(&so.ml_full), peer));
      }
    }
  } else {
    if (warp == 0) {
      // ---------------------------------------------------- V loads (CTA 1)
      if (lane == 0) {
        int vc = 0;
        for (; next_piece(false); ++pieces) {
          // table entries are loaded a tile before they are used
          int e0 = unit_entry(A, x, 2 * p.t0), e1 = unit_entry(A, x, 2 * p.t0 + 1);
          for (int t = p.t0; ok && t < p.t1; ++t) {
            const int n = tile_units(x, t);
            const int c0 = entry_row(A, e0), c1 = entry_row(A, e1);
            e0 = unit_entry(A, x, 2 * t + 2);
            e1 = unit_entry(A, x, 2 * t + 3);
            for (int h = 0; h < 2 * n; ++h, ++vc) {
              const int st = vc & 3;
              if (vc >= kVRing &&
                  !(ok = wait1(so.v_empty[st], ((vc >> 2) + 1) & 1, abort_flag, err)))
                break;
              const uint32_t full = smem_u32(&so.v_full[st]);
              mbar_expect_tx(full, kVChunk);
              tma_load_3d(smem_u32(so.v[st]), &tm_v, full, 0, h < 2 ? c0 : c1, 4 * (h & 1));
            }
          }
        }
        if (!ok)
          for (int c = max(0, vc - kVRing); c < vc; ++c)
            mbar_drain(smem_u32(&so.v_full[c & 3]), (c >> 2) & 1);
      }
    } else if (warp == 1) {
      // ------------------------------------------------------- PV (CTA 1)
      // One thread.
      if (elect_one()) {
        const uint32_t id = idesc_bf16(128, 256, true);
        const uint64_t p_d = sdesc_sw128(smem_u32(so.p[0]), 0, 1024);
        const uint64_t v_d = sdesc_sw128(smem_u32(so.v[0]), kUnitAtom, 1024);
        int vc = 0, tc = 0, ac = 0;
        unsigned cleaned = 0;                           // parity of each unit's uses of `clean`
        for (; next_piece(false); ++pieces) {
          for (int t = p.t0; ok && t < p.t1; ++t, ++tc) {
            const int n = tile_units(x, t);
            if (!(ok = wait1(so.o_ok[tc & 3], (tc >> 2) & 1, abort_flag, err))) break;
            tc_fence_after();
            for (int u = 0; ok && u < n; ++u, ++ac) {
              const int slot = ac & 3;
              if (!(ok = wait1<true>(so.p_full[slot], (ac >> 2) & 1, abort_flag, err))) break;
              if (2 * t + u < x.nu && unit_hidden(A, x, 2 * t + u) != 0ull) {
                if (!(ok = wait1(so.clean[u], (cleaned >> u) & 1, abort_flag, err))) break;
                cleaned ^= 1u << u;
              }
              const uint64_t pd = p_d + slot * (kAtom >> 4);
#pragma unroll 1
              for (int h = 0; h < 2; ++h, ++vc) {
                const int st = vc & 3;
                if (!(ok = wait1(so.v_full[st], (vc >> 2) & 1, abort_flag, err))) break;
                const uint64_t vd = v_d + st * (kVChunk >> 4);
#pragma unroll
                for (int kk = 0; kk < 4; ++kk)          // 16 keys: 32 B of P, 2 KB of V
                  mma_bf16(tmem + 256 * h, pd + 2 * kk, vd + (kk * 2048 >> 4), id,
                           (t > p.t0 || u > 0 || kk > 0) ? 1u : 0u);
                mma_commit(smem_u32(&so.v_empty[st]));
              }
              mma_commit(smem_u32(&so.p_free[slot]));
            }
            mma_commit(smem_u32(&so.pv_done[tc & 3]));
            abort_flag[1] = tc;
          }
          mma_commit(smem_u32(&ctl.o_done));
        }
        if (!ok) {
          mma_commit(smem_u32(&ctl.q_free));
          mbar_drain(smem_u32(&ctl.q_free), 0);
        }
      }
      __syncwarp();
    } else if (warp == 2 || warp == 3) {
      // ---- word to CTA 0: an atom has landed (warp 2), its slot is free (warp 3)
      if (lane == 0) {
        int a = 0, tc = 0;
        for (; next_piece(false); ++pieces) {
          for (int t = p.t0; ok && t < p.t1; ++t, ++tc) {
            const int n = tile_units(x, t);
#pragma unroll 1
            for (int u = 0; u < n; ++u, ++a) {
              const int slot = a & 3;
              if (warp == 2) {
                if (u == 0 &&
                    !(ok = wait1<true>(so.al_full[tc & 3], (tc >> 2) & 1, abort_flag, err)))
                  break;
                if (!(ok = wait1<true>(so.p_full[slot], (a >> 2) & 1, abort_flag, err))) break;
                mbar_arrive_remote(mapa(smem_u32(&ctl.p_ack[tc & 1][u]), peer));
              } else {
                if (!(ok = wait1(so.p_free[slot], (a >> 2) & 1, abort_flag, err))) break;
                mbar_expect_tx(smem_u32(&so.p_full[slot]), kAtom);
                mbar_arrive_remote(mapa(smem_u32(&ctl.p_room[slot]), peer));
              }
            }
          }
        }
      }
    } else if (warp == 13) {
      // -------------------------------------------- the pieces (CTA 1)
      // Piece k is written once the output of piece k - 4 is on its way. The
      // place it takes was piece k - 8's, which every role has copied by then:
      // no role is more than four atoms of P behind the output, and a piece
      // has at least one.
      for (pieces = 1; p.item >= 0; ++pieces) {
        const int done = pieces - kPieces / 2;
        if (!(ok = ok && (done < 0 || wait32(so.piece_done[done & (kPieces - 1)],
                                             (done / kPieces) & 1, abort_flag, err))))
          break;
        p = walk.next(A);
        const int slot = pieces & (kPieces - 1);
        if (lane == 0) ctl.piece[slot] = p;
        __syncwarp();
        if (lane < static_cast<int>(sizeof(Piece) / 4)) {
          const float* w = reinterpret_cast<const float*>(&ctl.piece[slot]) + lane;
          st_cluster_f32(mapa(smem_u32(w), peer), *w);
        }
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(smem_u32(&ctl.piece_full[slot]));
          mbar_arrive_remote(mapa(smem_u32(&ctl.piece_full[slot]), peer));
        }
      }
    } else if (warp < 12) {
      // ------------------------------------- rescale and output (CTA 1)
      const int g = (warp - 4) >> 2;                    // half of the 512 value dims
      const int wq = warp & 3;
      const int r = 32 * wq + lane;
      const uint32_t o_cols = tmem + (static_cast<uint32_t>(32 * wq) << 16) + 256 * g;
      int tc = 0, vc = 0;
      bool recorded = false;
      // a long piece's second sum: the place of its part, or of the next one
      float scale = 1.f;
      auto sum = [&]() {
        return A.part_o + (2ll * cluster + (p.first ? 1 : 0)) * 128 * A.rows_pad +
               64ll * g * A.rows_pad + r;
      };
      for (; next_piece(true); ++pieces) {
        for (int t = p.t0; ok && t < p.t1; ++t, ++tc) {
          const int n = tile_units(x, t);
          const int sl4 = tc & 3;
          if (!(ok = wait32<true>(so.al_full[sl4], (tc >> 2) & 1, abort_flag, err))) break;
          if (threadIdx.x == 128) mbar_expect_tx(smem_u32(&so.al_full[sl4]), 512);
          const float alpha = so.alpha[sl4][r];
          const int age = t - p.t0;
          const bool full = age > 0 && age % kSumTiles == 0;
          if (age > kSumTiles) scale *= alpha;
          if (__any_sync(0xffffffffu, alpha != 1.f) || full) {
            // never on a piece's first tile, so the PV of the tile before is this piece's
            if (!(ok = wait32(so.pv_done[(tc + 3) & 3], ((tc - 1) >> 2) & 1, abort_flag, err)))
              break;
            tc_fence_after();
#pragma unroll 1
            for (int cc = 0; cc < 8; ++cc) {
              float o[32];
              tmem_ld32(o_cols + 32 * cc, o);
#pragma unroll
              for (int e = 0; e < 32; ++e) o[e] *= alpha;
              tmem_st32(o_cols + 32 * cc, o);
            }
            if (full) {
              move_sum(sum(), A.rows_pad, r < x.nrows, scale, age == kSumTiles, false, o_cols);
              scale = 1.f;
            }
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(&so.o_ok[sl4]));
          // Keys that some row does not see have zeros in its P, and a zero
          // times a NaN or infinite value would reach that row: such values
          // become 0, and the rows that see them get theirs at the end. PV of
          // this unit waits for `clean`.
          for (int u = 0; u < n; ++u, vc += 2) {
            const unsigned long long hidden =
                2 * t + u < x.nu ? unit_hidden(A, x, 2 * t + u) : 0ull;
            if (hidden == 0ull) continue;
            // once the tile before is done, its chunks' barriers are in the
            // phase before the one waited for
            if (t > p.t0 && !(ok = wait32(so.pv_done[(tc + 3) & 3], ((tc - 1) >> 2) & 1,
                                          abort_flag, err)))
              break;
            const int k0 = __ffsll(static_cast<long long>(hidden)) - 1;
            const int k1 = 64 - __clzll(static_cast<long long>(hidden));
            for (int h = 0; h < 2; ++h) {
              const int c = vc + h;
              if (!(ok = wait32(so.v_full[c & 3], (c >> 2) & 1, abort_flag, err))) break;
              uint8_t* v = so.v[c & 3];
              const int sub = static_cast<int>(threadIdx.x) - 128;
              unsigned bad = 0;
#pragma unroll 2
              for (int i = sub >> 3; i < 4 * (k1 - k0); i += kCleaners / 8) {
                const uint4 o = *v_piece(v, k0, i, sub);
                bad |= not_finite(o.x) | not_finite(o.y) | not_finite(o.z) | not_finite(o.w);
              }
              if (bad)
                clean_v(A, v, k0, k1, sub, unit_block(x, 2 * t + u) * 64, 256 * h, x.pos0, x.last,
                        x.nrows, so.lost, so.o_ok[sl4], (tc >> 2) & 1, abort_flag, err);
            }
            if (!ok) break;
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&so.clean[u]));
          }
        }
        if (!ok) break;
        // ------------------------------------------------------- a piece's end
        if (!(ok = wait32<true>(so.ml_full, pieces & 1, abort_flag, err))) break;
        const float2 a0 = so.ml[0][r], a1 = so.ml[1][r];
        __syncwarp();
        if (lane == 0) mbar_arrive_remote(mapa(smem_u32(&ctl.ml_free), peer));
        const float m = fmaxf(a0.x, a1.x);
        const float l = (a0.x > -INFINITY ? a0.y * fast_exp2(a0.x - m) : a0.y) +
                        (a1.x > -INFINITY ? a1.y * fast_exp2(a1.x - m) : a1.y);
        if (!(ok = wait32(ctl.o_done, pieces & 1, abort_flag, err))) break;
        tc_fence_after();
        if (p.t1 - p.t0 > kSumTiles)
          move_sum(sum(), A.rows_pad, r < x.nrows, scale, false, true, o_cols);
        const uint4 lost0 = *reinterpret_cast<const uint4*>(&so.lost[r][8 * g]);
        const uint4 lost1 = *reinterpret_cast<const uint4*>(&so.lost[r][8 * g + 4]);
        if (__any_sync(0xffffffffu, (lost0.x | lost0.y | lost0.z | lost0.w | lost1.x | lost1.y |
                                     lost1.z | lost1.w) != 0u))
          spoil_lost(&so.lost[r][8 * g], o_cols);
        const bool valid = r < x.nrows;
        if (p.first && p.last) {
          const float inv = l == 0.f ? 0.f : 1.f / l;
          // 32 dims at a time through shared memory (row of 64 B, 16-B chunk c
          // at c ^ (row / 2 % 4)), so that a warp's store covers whole sectors
          uint8_t* mine = so.stage[warp - 4];
          const int sub = lane & 3, row0 = lane >> 2;
          __nv_bfloat16* out = A.out + (x.row0 + 32 * wq) * 512 + 256 * g + 8 * sub;
#pragma unroll 1
          for (int cc = 0; cc < 8; ++cc) {
            float o[32];
            tmem_ld32(o_cols + 32 * cc, o);
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              uint32_t w[4];
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const __nv_bfloat162 v = __floats2bfloat162_rn(o[8 * c + 2 * e] * inv,
                                                               o[8 * c + 2 * e + 1] * inv);
                w[e] = *reinterpret_cast<const uint32_t*>(&v);
              }
              *reinterpret_cast<uint4*>(mine + lane * 64 + ((c ^ ((lane >> 1) & 3)) << 4)) =
                  make_uint4(w[0], w[1], w[2], w[3]);
            }
            __syncwarp();
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const int row = row0 + 8 * k;
              const uint4 v = *reinterpret_cast<const uint4*>(
                  mine + row * 64 + ((sub ^ ((row >> 1) & 3)) << 4));
              if (32 * wq + row < x.nrows)
                *reinterpret_cast<uint4*>(out + static_cast<long long>(row) * 512 + 32 * cc) = v;
            }
            __syncwarp();
          }
          if (g == 0 && valid && A.lse)
            A.lse[x.row0 + r] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.69314718055994531f;
        } else {
          // one of the parts of a cut row tile: slot 1 of the cluster that
          // holds its first tile, slot 0 of the others
          const long long slot = 2 * cluster + (p.first ? 1 : 0);
          float4* po = A.part_o + slot * 128 * A.rows_pad + r;
#pragma unroll 1
          for (int cc = 0; cc < 8; ++cc) {
            float o[32];
            tmem_ld32(o_cols + 32 * cc, o);
            if (!valid) continue;
#pragma unroll
            for (int e = 0; e < 8; ++e)
              po[static_cast<long long>(64 * g + 8 * cc + e) * A.rows_pad] =
                  make_float4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
          }
          if (g == 0 && valid) A.part_ml[slot * A.rows_pad + r] = make_float2(m, l);
          if (p.first && threadIdx.x == 128) {
            const long long at = p.start + kItemCost + x.tiles - 1;
            const long long total = ctl.share.total;
            const int parts = ctl.share.parts;
            int e = static_cast<int>(at * parts / total);
            while (e + 1 < parts && share_begin(total, parts, e + 1) <= at) ++e;
            while (e > 0 && share_begin(total, parts, e) > at) --e;
            A.rec[cluster] = make_int2(p.item, e);
            recorded = true;
          }
        }
        if (threadIdx.x == 128)
          mbar_arrive(smem_u32(&so.piece_done[pieces & (kPieces - 1)]));
      }
      if (threadIdx.x == 128 && !recorded && A.rec) A.rec[cluster] = make_int2(-1, 0);
    }
  }
  tc_fence_before();
  __syncwarp();
  cluster_sync();          // the peer no longer touches this CTA's shared memory
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// Joins the parts of the cut row tiles. Record c names the row tile whose first
// tile closes cluster c's share; a cluster that ran nothing, or gave up before it
// wrote a first part, leaves none. So the error word, which other streams set and
// clear, is not looked at here: what the first launch wrote is joined. A task is
// 32 rows and 128 value dims of a row tile, 16 dims a warp; where the row tile has
// many parts, 8 dims, whose parts the eight warps share. The weights are worked
// out once a task. A warp reads 512 consecutive bytes at a time (four dims of 32
// rows), eight reads in flight, the first of them asked for before the weights are
// known. Bound by the latency of a task's chain (record, maxima, weights, sums), so
// tasks are few and large: one sequence of 131072 tokens, 73 parts of 256 KB, 7 us
// with the launch (13 us in tasks of 32 dims with the weights worked out for each);
// 33 sequences of up to 32768, two queries each, 9 us (20 us).
constexpr int kJoinThreads = 256, kJoinResident = 3, kJoinCtas = kJoinResident * 148;
constexpr int kJoinBatch = (kMaxClusters + 7) / 8;              // parts a warp weighs
constexpr int kJoinRecs = (kMaxClusters + 31) / 32;             // records a lane looks at
// Parts from which the warps share them (33 ragged sequences, two queries each:
// 95 us with 16, 97 us with 8; one of 131072 tokens has 73 and is the same).
constexpr int kJoinMany = 16;
constexpr int kJoinFewDims = 4, kJoinManyDims = 2;              // a warp's dims, in fours
struct JoinSmem {
  float weight[kMaxClusters][32];
  float top[8][32], sum[8][32];
  float4 partial[8][kJoinManyDims][32];
};
__device__ __forceinline__ int join_tasks(int parts) {          // of 32 rows
  return parts > kJoinMany ? 128 / kJoinManyDims : 128 / (8 * kJoinFewDims);
}
// One task: dims 4 c4 .. 4 (c4 + kDims) of 32 rows for this warp, its parts [i0, i1).
template <int kDims, bool kShared>
__device__ __forceinline__ void join_rows(JoinSmem& sj, const RangeArgs& A, long long row, bool valid,
                                          int r, int c, int n, int c4, int i0, int i1) {
  constexpr int kStep = 8 / kDims;              // parts at a time
  const int warp = warp_id(), lane = lane_id();
  auto slot = [&](int i) { return static_cast<long long>(2 * (c + i) + (i == 0 ? 1 : 0)); };
  const long long pitch = 128ll * A.rows_pad;
  const float4* part = A.part_o + static_cast<long long>(c4) * A.rows_pad + r;
  float4 v[8];
  auto fetch = [&](int i) {
#pragma unroll
    for (int k = 0; k < 8; ++k)
      v[k] = valid && i + k / kDims < i1
                 ? part[slot(i + k / kDims) * pitch + (k % kDims) * A.rows_pad]
                 : make_float4(0.f, 0.f, 0.f, 0.f);
  };
  float2 ml[kJoinBatch];
#pragma unroll
  for (int k = 0; k < kJoinBatch; ++k) {
    const int i = warp + 8 * k;
    ml[k] = valid && i < n ? A.part_ml[slot(i) * A.rows_pad + r] : make_float2(-INFINITY, 0.f);
  }
  fetch(i0);
  float m = -INFINITY, l = 0.f;
#pragma unroll
  for (int k = 0; k < kJoinBatch; ++k) m = fmaxf(m, ml[k].x);
  __syncthreads();                              // the task before is done with the tables
  sj.top[warp][lane] = m;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < 8; ++w) m = fmaxf(m, sj.top[w][lane]);
  const float base = m == -INFINITY ? 0.f : m;
#pragma unroll
  for (int k = 0; k < kJoinBatch; ++k) {
    const int i = warp + 8 * k;
    if (i >= n) continue;
    const float w = fast_exp2(ml[k].x - base);
    sj.weight[i][lane] = w;
    l += ml[k].x == -INFINITY ? ml[k].y : w * ml[k].y;          // (a NaN sum of a part stays one)
  }
  sj.sum[warp][lane] = l;
  __syncthreads();
  float4 o[kDims] = {};
  auto add = [](float4& s, const float4& a, float w) {
    s.x += w * a.x;
    s.y += w * a.y;
    s.z += w * a.z;
    s.w += w * a.w;
  };
  for (int i = i0; i < i1;) {
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (i + k / kDims < i1) add(o[k % kDims], v[k], sj.weight[i + k / kDims][lane]);
    i += kStep;
    if (i < i1) fetch(i);
  }
  if constexpr (kShared) {
#pragma unroll
    for (int d = 0; d < kDims; ++d) sj.partial[warp][d][lane] = o[d];
    __syncthreads();
    if (warp != 0) return;
    for (int w = 1; w < 8; ++w) {
#pragma unroll
      for (int d = 0; d < kDims; ++d) add(o[d], sj.partial[w][d][lane], 1.f);
    }
  }
  if (!valid) return;
  l = 0.f;
#pragma unroll
  for (int w = 0; w < 8; ++w) l += sj.sum[w][lane];
  const float inv = l == 0.f ? 0.f : 1.f / l;
  uint32_t w[2 * kDims];
#pragma unroll
  for (int d = 0; d < kDims; ++d) {
    const __nv_bfloat162 a = __floats2bfloat162_rn(o[d].x * inv, o[d].y * inv);
    const __nv_bfloat162 b = __floats2bfloat162_rn(o[d].z * inv, o[d].w * inv);
    w[2 * d] = *reinterpret_cast<const uint32_t*>(&a);
    w[2 * d + 1] = *reinterpret_cast<const uint32_t*>(&b);
  }
  uint4* out = reinterpret_cast<uint4*>(A.out + row * 512 + 4 * c4);
#pragma unroll
  for (int d = 0; d < kDims / 2; ++d)
    out[d] = make_uint4(w[4 * d], w[4 * d + 1], w[4 * d + 2], w[4 * d + 3]);
  if (c4 == 0 && A.lse)
    A.lse[row] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.69314718055994531f;
}
__global__ void __launch_bounds__(kJoinThreads, kJoinResident)
range_join_kernel(const __grid_constant__ RangeArgs A) {
  __shared__ JoinSmem sj;
  const int warp = warp_id(), lane = lane_id();
  const int row_blocks = (A.rows_pad + 31) >> 5;
  // the records' tasks, laid end to end: this lane's end at `end`
  int item[kJoinRecs], parts[kJoinRecs], tasks = 0;
#pragma unroll
  for (int k = 0; k < kJoinRecs; ++k) {
    const int c = kJoinRecs * lane + k;
    const int2 rec = c < A.clusters ? A.rec[c] : make_int2(-1, 0);
    item[k] = rec.x;
    parts[k] = rec.y - c + 1;                   // slot 1 of c, slot 0 of c+1 .. rec.y
  }
#pragma unroll
  for (int k = 0; k < kJoinRecs; ++k)
    if (item[k] >= 0) tasks += join_tasks(parts[k]) * row_blocks;
  int end = tasks;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, end, o);
    if (lane >= o) end += y;
  }
  const int total = __shfl_sync(0xffffffffu, end, 31);
  for (int task = static_cast<int>(blockIdx.x); task < total; task += kJoinCtas) {
    const int owner = __ffs(__ballot_sync(0xffffffffu, task < end)) - 1;
    int at = task - (end - tasks), c = 0, it = 0, n = 0;
#pragma unroll
    for (int k = 0; k < kJoinRecs; ++k) {
      if (item[k] < 0 || n) continue;
      const int t = join_tasks(parts[k]) * row_blocks;
      if (at < t) {
        c = kJoinRecs * lane + k;
        it = item[k];
        n = parts[k];
      } else {
        at -= t;
      }
    }
    at = __shfl_sync(0xffffffffu, at, owner);
    c = __shfl_sync(0xffffffffu, c, owner);
    it = __shfl_sync(0xffffffffu, it, owner);
    n = __shfl_sync(0xffffffffu, n, owner);
    const int b = it / A.per_seq, j0 = (it - b * A.per_seq) * A.G;
    const int nq = A.block_table ? A.nq : A.T;
    const int across = join_tasks(n), block = at / across, group = at - block * across;
    const int r = 32 * block + lane;
    const bool valid = r < min(A.G, nq - j0) * A.H;
    const long long row = (static_cast<long long>(b) * nq + j0) * A.H + r;
    if (n > kJoinMany)
      join_rows<kJoinManyDims, true>(sj, A, row, valid, r, c, n, kJoinManyDims * group,
                                     n * warp / 8, n * (warp + 1) / 8);
    else
      join_rows<kJoinFewDims, false>(sj, A, row, valid, r, c, n, kJoinFewDims * (8 * group + warp),
                                     0, n);
  }
}

}  // namespace

size_t range_layout(RangeArgs& a, void* workspace) {
  const int queries = a.block_table ? a.nq : a.T;
  a.G = std::max(1, std::min(queries, 128 / a.H));
  a.per_seq = (queries + a.G - 1) / a.G;
  const long long items = (a.block_table ? static_cast<long long>(a.B) : 1ll) * a.per_seq;
  a.items = static_cast<int>(items);
  // tiles a row tile can have
  const long long keys = a.block_table ? static_cast<long long>(a.max_blocks) * 64 : a.S;
  long long units = (keys + 63) / 64;
  if (a.window)
    units = std::min(units, (static_cast<long long>(a.window) + a.G + 63) / 64 + 1 +
                                (std::min<long long>(a.sinks, keys) + 63) / 64);
  const long long tiles = (units + 1) / 2;
  a.whole = !a.block_table && items > kScanItems;
  a.clusters = static_cast<int>(std::min<long long>(kMaxClusters, items * (tiles + kItemCost)));
  a.rows_pad = (a.G * a.H + 7) / 8 * 8;
  a.rec = nullptr;
  a.part_ml = nullptr;
  a.part_o = nullptr;
  if (a.whole && tiles <= kSumTiles) return 0;
  auto up = [](size_t v) { return (v + 255) / 256 * 256; };
  const size_t n = static_cast<size_t>(a.clusters);
  const size_t rec = up(n * sizeof(int2)), ml = up(2 * n * a.rows_pad * sizeof(float2));
  const size_t parts = 2 * n * 128 * a.rows_pad * sizeof(float4);
  char* ws = static_cast<char*>(workspace);
  if (a.whole) {                                // no row tile is cut: second sums only
    a.part_o = reinterpret_cast<float4*>(ws);
    return parts;
  }
  a.rec = reinterpret_cast<int2*>(ws);
  a.part_ml = ws ? reinterpret_cast<float2*>(ws + rec) : nullptr;
  a.part_o = ws ? reinterpret_cast<float4*>(ws + rec + ml) : nullptr;
  return rec + ml + parts;
}

cudaError_t launch_range_mla(const RangeArgs& a_in, cudaStream_t st) {
  RangeArgs a = a_in;
  a.kv_rows = a.block_table ? a.nblk * 64 : a.S;
  const long long q_rows = (a.block_table ? static_cast<long long>(a.B) * a.nq : a.T) * a.H;
  CUtensorMap tq, tk, tv;
  cudaError_t e = make_tmap_2d(&tq, a.q, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 576, q_rows, 576 * 2,
                               64, 128, CU_TENSOR_MAP_SWIZZLE_128B);
  if (e == cudaSuccess) e = make_tmap_chunks(&tk, a.kv, a.kv_rows, 64, 1);
  if (e == cudaSuccess) e = make_tmap_chunks(&tv, a.kv, a.kv_rows, 64, 4);
  if (e != cudaSuccess) return e;
  e = cudaFuncSetAttribute(range_mla_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           static_cast<int>(kSmemBytes));
  if (e != cudaSuccess) return e;
  range_mla_kernel<<<2 * a.clusters, kThreads, kSmemBytes, st>>>(tq, tk, tv, a);
  e = cudaGetLastError();
  if (e != cudaSuccess || !a.rec) return e;
  range_join_kernel<<<kJoinCtas, kJoinThreads, 0, st>>>(a);
  return cudaGetLastError();
}

}  // namespace dsa
