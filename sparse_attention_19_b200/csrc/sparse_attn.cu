// sparse_attn.cu -- sparse MQA / MLA-absorbed attention over the selected latent rows.
//
// For query row r (batch b, position t) and head h, over the selected positions s:
//   z_s = scale * q[r,h,:] . kv[b,s,:]        (all d_qk columns: latent + rope)
//   out[r,h,:] = sum_s softmax(z)_s * kv[b,s,:d_v]
// (DeepSeek-V3.2 technical-report summary, "Отбор и основное внимание", equation
// for u_t: attention only over the top-k latent entries c_s; MLA in MQA mode, one
// KV row serves every query head.)
//
// Mapping onto a pair of SMs (a 2-CTA cluster, tcgen05 .cta_group::2):
//   * Each CTA owns 64 of the 128 query heads; its Q rows (64 x d_qk bf16) stay in
//     shared memory for the whole query.  MMA M = 128 heads across the pair.
//   * Keys come in tiles of 128 selected positions.  S = Q K^T is one pair-MMA
//     chain with N = 128 keys: each CTA gathers 64 of the tile's key rows, in
//     64-column chunks (TMA tile::gather4, 128-byte swizzle), streamed through a
//     ring.  S lands in TMEM as 64 columns per CTA (lanes 0-63: keys 0-63,
//     lanes 64-127: keys 64-127 of the tile, for that CTA's 64 heads).
//   * Four softmax warps per CTA turn S into P (bf16, in shared memory, the A
//     operand of the next MMA) with an online softmax whose reference maximum
//     only moves when a new maximum exceeds it by 2^8 (the accumulator is then
//     rescaled in TMEM); the two lanes that hold one head's two key halves swap
//     their maxima through shared memory.
//   * O += P V is a pair-MMA with N = 256 value columns per instruction; V is
//     the same gathered rows read as an MN-major operand, each CTA holding 128
//     value columns of all 128 keys.  O for 64 heads x 512 columns fits in 256
//     TMEM columns per CTA (the pair layout puts half of N in lanes 64-127), so
//     S double-buffers beside it.
//   * The leader CTA (rank 0) issues every MMA; both CTAs' TMA loads complete on
//     the leader's barriers, and MMA completion is multicast to both CTAs.  The
//     softmax warps of both CTAs signal the leader's barriers directly (after a
//     fence.proxy.async for the P tile they wrote).  P is double-buffered, so the
//     softmax of tile j+1 overlaps the P.V of tile j.
//   * S = Q K^T and O += P V are issued by two threads (warps 4 and 5 of the
//     leader): at these shapes one thread's issue rate, not the tensor core, would
//     bound the MMAs, and P.V(j) then never waits behind the key chunks of S(j+1).
//   * Loads: TMA requests from one warp are served in order, so the gather rate
//     grows with the number of issuing warps.  Key chunks come from 9 warps and
//     value stages from 9 others (each group walks its own ring, so a value slot
//     that is still in use never holds back the next tile's keys); the value
//     loaders also stage each unit's selected positions, one unit ahead.
// Warp roles (768 threads per CTA): warps 0-3 softmax/epilogue (TMEM lane quarter
// = warp), warp 4 TMEM owner + S issuer (leader), warp 5 P.V issuer (leader),
// warps 6-14 key loaders, warps 15-23 value loaders + index staging.  The softmax
// warpgroup holds 120 registers per thread, the others 72 (setmaxnreg).
//
// The kernel has two more forms that differ in where the keys come from (AttnMode below):
//   * a sliding window and sinks (kWindow): the slots of a row are computed, not listed; 16
//     slots that are consecutive rows come in one box (68 TMA requests a tile and CTA instead of 272), a group
//     with the seam or the end of the row by gathers.  Rows past the query or between the sinks
//     and the window are never loaded, since a zero probability times a NaN would still
//     reach the output.  4096 rows x (512 + 16) slots 857 us among other passes (703 TFLOP/s on the
//     slots, 0.43 of the bf16 burst peak), 735 alone at burst clocks (0.50); bound by the chain
//     S -> softmax -> P.V over only five tiles per row, the last of them one eighth full.
//   * rows of the 4-bit cache (kPacked): 16 warps convert codes to bf16 planes in shared
//     memory, in the layouts TMA writes for bf16 rows, once as key chunks and once as
//     value stages.  Everything behind the operands is shared, so the result equals the bf16
//     kernel's over the values that the cache holds bit for bit.  64 rows x 2048 68 us (bf16 rows 65:
//     the cache saves memory, not time).  Meant for rows used a few times
//     (decode); a chunk of queries that use each row many times has the cache unpacked first and runs
//     kSelected, with masked slots gathering a row of zeros (the host's rule has the figures).
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>

#include "dsa_internal.h"
#include "kv4.cuh"
#include "ptx.cuh"

namespace dsa {

namespace {

constexpr int kTileKeys = 128;       // keys per tile (pair)
constexpr int kHalfKeys = 64;        // keys per CTA in S, and keys per V stage
constexpr int kPBufs = 2;            // P buffers (2 planes each: keys 0-63, 64-127)
constexpr int kMaxIdx = 2048;        // selected positions per unit (staged in shared memory)
constexpr int kMmaWarp = 4;           // TMEM owner + S issuer
constexpr int kPvWarp = 5;            // P.V issuer
// Where the keys come from.
enum AttnMode {
  kSelected = 0,   // bf16 rows picked by an index list (or, dense, rows 0..t)
  kWindow = 1,     // bf16 rows of a sliding window and the first `sinks` positions
  kPacked = 2      // rows of the 4-bit cache picked by an index list
};
// Rings, loader warps and registers of a mode.
//
// kSelected, kWindow: loaders own ring slots, so a warp waits only on its own slots
// (in ring order) and the stages of different slots are issued in parallel.  Key
// chunks: a team of kKTeamWarps warps owns kKTeamSlots consecutive slots and splits
// each chunk's 16 gathers; value stages: kVWarpsPerSlot warps per slot split its gathers.
// A window's rows are mostly contiguous (boxes of 16 rows instead of gathers of 4), so
// one warp per slot issues fast enough; that leaves room for a fourth value stage
// (it also needs no staged index lists) and for 128 registers in every thread.
//
// kPacked: 16 loader warps convert; they read the index lists themselves (two warps only
// stage the validity words), and the room of the staged lists goes to a fourth value stage
// (two more key slots instead: 798 against 772 us on 1024 rows x 2048 keys).
//
// Register split: a CTA of 768 threads launches with 80 registers per thread (6 warps
// per SM sub-partition); the softmax warpgroup then takes 120 and the other
// warpgroups (MMA issuers, loaders) keep 72.
template <int MODE>
struct Cfg {
  static constexpr int kKStages = 6;                   // K-chunk ring depth (8 KB stages)
  static constexpr int kVStages = MODE == kSelected ? 3 : 4;   // V ring depth (64 keys x this CTA's value planes)
  static constexpr int kKTeamWarps = MODE == kWindow ? 1 : 3;
  static constexpr int kKTeamSlots = MODE == kWindow ? 1 : 2;
  static constexpr int kVWarpsPerSlot = MODE == kWindow ? 1 : 3;
  static constexpr int kKWarp0 = MODE == kPacked ? 8 : 6;   // key-chunk loaders
  static constexpr int kKWarps = MODE == kPacked ? 8 : kKStages / kKTeamSlots * kKTeamWarps;
  static constexpr int kVWarp0 = kKWarp0 + kKWarps;    // value-stage loaders
  static constexpr int kVWarps = MODE == kPacked ? 8 : kVStages * kVWarpsPerSlot;
  static constexpr int kThreads = 32 * (kVWarp0 + kVWarps);   // 768 (kWindow: 512)
  static constexpr int kStageWarps = MODE == kPacked ? 2 : kVWarps;   // warps that stage the indices
  // Arrivals that fill a key slot and a value slot (kPacked: 8 warps, or a team of 4 twice, and a
  // team, of both CTAs).
  static constexpr int kKFillers = MODE == kPacked ? 16 : 1, kVFillers = MODE == kPacked ? 8 : 1;
  static constexpr int kIdxReaders = MODE == kPacked ? 0 : kKWarps + kVWarps;   // loader warps that read staged indices
  static constexpr bool kSplitRegs = kThreads > 512;
};
static_assert(Cfg<kPacked>::kKWarps == 8 && Cfg<kPacked>::kVWarps == 8, "two teams of four warps each");
constexpr int kMaxKStages = 6, kMaxVStages = 4;
constexpr int kStageBatch = 8;       // index words in flight per warp while staging
constexpr uint32_t kRegsLaunch = 80;
constexpr uint32_t kRegsSoftmax = 120;
constexpr uint32_t kRegsOther = 72;
static_assert(128 * kRegsSoftmax + (768 - 128) * kRegsOther <= 768 * kRegsLaunch,
              "register split exceeds the launch allocation");
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kPlane64 = 64 * 128;    // 64 rows x 128 B  (Q plane, K stage, V plane, P plane)
constexpr uint32_t kTmemS = 0;             // S buffers: columns [0, 128)
constexpr uint32_t kTmemO = 128;           // O: columns [128, 128 + d_v/2)
constexpr float kRescaleThreshold = 8.0f;  // log2 units
constexpr float kLn2 = 0.6931471805599453f;
constexpr int kMaxChunks = 9;

struct AttnBarriers {
  uint64_t q_full[kMaxChunks], q_empty[kMaxChunks];
  uint64_t k_full[kMaxKStages], k_empty[kMaxKStages];
  uint64_t v_full[kMaxVStages], v_empty[kMaxVStages];
  uint64_t s_full[2], s_empty[2];
  uint64_t p_full[kPBufs], p_empty[kPBufs];
  uint64_t o_full, o_empty, final_s, final_pv;
  uint64_t idx_full[2], idx_empty[2];
  uint32_t valid_mask[2][kMaxIdx / 32];   // per 32 staged positions: bit set = valid entry
  uint64_t xbar[2];          // rendezvous of softmax warps w and w ^ 2 (same heads, other key half)
  uint32_t tmem_base;
  uint32_t abort_flag;
  float red_max[2][128];
  float red_sum[128];
};

template <int DV>
struct VShape {
  static constexpr int kNpv = DV >= 256 ? DV / 256 : 1;   // PV instructions per tile
  static constexpr int kN = DV >= 256 ? 256 : DV;         // N of one PV instruction
  static constexpr int kPlanes = kN / 128;                // 64-column planes per CTA per instruction
  static constexpr uint32_t kStageBytes = kPlanes * kPlane64;   // 64 keys x planes
};

// A unit is one query row's key-tile range [j0, j1) (the whole row without split-k).
struct Unit {
  int row, b, t, j0, j1, split;
  int n_sinks, lo, n_valid;   // kWindow: slots 0..n_sinks-1 are keys 0.., the others keys lo..; n_valid slots
};

template <int MODE>
__device__ __forceinline__ Unit decode_unit(const AttnParams& p, int u) {
  Unit U;
  const int n_rows = p.B * p.Lq;
  U.row = n_rows - 1 - u / p.splits;       // longest rows first (top-k output is valid-first)
  U.split = u % p.splits;
  U.b = U.row / p.Lq;
  U.t = p.q_offset + U.row % p.Lq;
  int nt = p.n_tiles;
  if constexpr (MODE == kWindow) {
    // Query position t sees keys max(0, t - window + 1) .. t and 0 .. sinks - 1, all
    // below Lk; a position outside the sequence (a padded row's start) sees what of
    // that exists, possibly nothing.
    const long long t = (long long)(p.start ? __ldg(p.start + U.b) : p.q_offset) + U.row % p.Lq;
    const long long lo = max(0ll, t - p.window + 1), hi = min(t, (long long)p.Lk - 1);
    U.n_sinks = (int)min(min((long long)p.sinks, lo), (long long)p.Lk);
    if (t < 0) U.n_sinks = 0;
    U.lo = (int)min(lo, (long long)p.Lk);
    U.n_valid = U.n_sinks + (int)max(0ll, hi - lo + 1);
    nt = (U.n_valid + kTileKeys - 1) / kTileKeys;
  } else if (p.compact) {
    const int nvalid = min(p.k, U.t + 1);
    nt = (nvalid + kTileKeys - 1) / kTileKeys;
  }
  U.j0 = min(nt, U.split * p.tiles_per_split);
  U.j1 = min(nt, (U.split + 1) * p.tiles_per_split);
  return U;
}

// First unit at or after u (stepping by the cluster count) that has key tiles;
// returns p.n_units when there is none.
template <int MODE>
__device__ __forceinline__ int next_unit(const AttnParams& p, int u, int step, Unit& U) {
  for (; u < p.n_units; u += step) {
    U = decode_unit<MODE>(p, u);
    if (U.j0 < U.j1) return u;
  }
  return p.n_units;
}

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<uint32_t*>(&v);
}

// Rows of kv (in the [B*Lk, d_qk] view) of four consecutive staged positions
// (pos a multiple of 4), one 16-byte shared-memory load; padding and out-of-range
// entries were staged as row b*Lk (a valid row), masked in the softmax.
__device__ __forceinline__ int4 gather_rows4(const int32_t* rows, int pos) {
  return *reinterpret_cast<const int4*>(rows + pos);
}

// kWindow: the key at slot x of a unit.  Slots behind the last valid one repeat it: their
// logits are masked, and a zero probability times a row that may hold anything (NaN) would
// still reach the output.
__device__ __forceinline__ int window_key(const Unit& U, int x) {
  x = min(x, U.n_valid - 1);
  return x < U.n_sinks ? x : U.lo + (x - U.n_sinks);
}

// kWindow: whether the unit's last tile has no valid slot in its second 64: then the values of
// that half, which would be multiplied by zeros, are neither loaded nor multiplied.
template <int MODE>
__device__ __forceinline__ bool one_half(const Unit& U) {
  return MODE == kWindow && U.n_valid - (U.j1 - 1) * kTileKeys <= kHalfKeys;
}

// kWindow: 64 rows (slots x0 ..) of 64 columns from column col into a plane, lanes 0-15,
// four rows each: one box per 16 rows that are consecutive keys, else gathers of four.
// Either way 8 KB complete on the barrier.
__device__ __forceinline__ void window_load(const AttnParams& p, const Unit& U, int x0, uint8_t* plane,
                                            const void* tmap_rows, const void* tmap_box, uint32_t bar, int col,
                                            int lane) {
  const int x = x0 + lane / 4 * 16, base = U.b * p.Lk;
  const int first = window_key(U, x);
  if (x >= U.n_valid && U.n_valid - U.n_sinks >= 16) {
    // nothing valid here: any 16 valid rows will do
    if (lane % 4 == 0) tma_load_2d_pair(plane + lane * 512, tmap_box, bar, col, base + U.lo);
  } else if (x + 15 < U.n_valid && window_key(U, x + 15) == first + 15) {
    if (lane % 4 == 0) tma_load_2d_pair(plane + lane * 512, tmap_box, bar, col, base + first);
  } else {
    const int y = x0 + lane * 4;
    tma_gather4_pair(plane + lane * 512, tmap_rows, bar, col, base + window_key(U, y), base + window_key(U, y + 1),
                     base + window_key(U, y + 2), base + window_key(U, y + 3));
  }
}

// 16 columns (two words) to the 16-byte columns at lo and hi of a swizzled row.
__device__ __forceinline__ void store_codes(uint8_t* row, uint32_t lo, uint32_t hi, uint32_t w0, uint32_t w1,
                                            uint32_t scale_bits) {
  const Kv4Step t = kv4_step(scale_bits);
  *reinterpret_cast<uint4*>(row + lo) = unpack_codes(w0, t);
  *reinterpret_cast<uint4*>(row + hi) = unpack_codes(w1, t);
}

// kPacked loaders.  Teams of four warps own alternate jobs: a job is 64 rows x 128 columns of
// 4-bit codes (two key chunks, or one value stage), 16 rows to a warp, four lanes to a row, 16
// columns of both chunks to a lane and row.  The registers that held a job's codes are
// loaded again for the next tile as soon as it is converted, so a tile of loads is in
// flight across units too.
// What sets the pace is the converting warps' instruction stream (times alone at burst clocks):
// without the conversions' arithmetic 861 -> 682 us (1024 rows x 2048 keys), without their loads 726, without their
// stores no gain, without all three 420.  So: one wait and one fence per job, not per chunk (822),
// the two chunks of a job in a rolled loop, since 24 warps in five roles also wait for
// instructions (754 -> 734); all eight warps in every chunk (986), one more team of key
// warps at 56 registers (923), or the tail chunk gathered by the staging warps (779) were slower.
struct TileCursor {
  Unit U;
  int u, j;               // unit (>= n_units: past the end) and tile
  const int32_t* list;    // the tile's index entries
  int left, base;         // entries of the list from there on; cache row of the sequence's row 0
  __device__ __forceinline__ void enter(const AttnParams& p) {
    j = U.j0;
    list = p.indices + (size_t)U.row * p.k + j * kTileKeys;
    left = u < p.n_units ? p.k - j * kTileKeys : 0;
    base = U.b * p.Lk;
  }
  __device__ __forceinline__ void start(const AttnParams& p, int cluster_id, int n_clusters) {
    u = next_unit<kPacked>(p, cluster_id, n_clusters, U);
    enter(p);
  }
  __device__ __forceinline__ void next(const AttnParams& p, int n_clusters) {
    if (u >= p.n_units) return;
    if (++j < U.j1) {
      list += kTileKeys;
      left -= kTileKeys;
    } else {
      u = next_unit<kPacked>(p, u + n_clusters, n_clusters, U);
      enter(p);
    }
  }
  // Entry x of the tile, as the cache row; -1 for a masked one.
  __device__ __forceinline__ int row(const AttnParams& p, int x) const {
    if (x >= left) return -1;
    int s;
    if (p.dense) {
      s = j * kTileKeys + x;
      if (s > U.t) return -1;
    } else {
      s = __ldg(list + x);
    }
    return (unsigned)s < (unsigned)p.Lk ? base + s : -1;
  }
};

// Key loaders.  Per tile, team t does chunk pairs t and t + 2, and each of the eight warps 8
// rows of the bf16 tail chunk.  Masked slots load some row: their logits are replaced.
template <int NC, int DV>
__device__ __forceinline__ void packed_keys(const AttnParams& p, AttnBarriers& S, uint8_t* k_sm, int pw,
                                            uint32_t rank, int cluster_id, int n_clusters,
                                            volatile uint32_t* abort_flag) {
  constexpr int kKStages = Cfg<kPacked>::kKStages;
  constexpr int kLat = DV / 64, kQ = kLat / 2;         // chunks of 4-bit columns, in pairs; then one bf16 tail chunk
  static_assert(NC == kLat + 1, "one tail chunk");
  constexpr int kPairs = (kQ + 1) / 2;                 // of a team
  const int lane = (int)lane_id(), r8 = lane / 4, part = lane % 4, team = pw / 4, w4 = pw % 4;
  const int x0 = (int)rank * kHalfKeys + w4 * 16 + r8;
  TileCursor c;
  c.start(p, cluster_id, n_clusters);
  if (c.u >= p.n_units) return;
  uint4 code[kPairs][2], tail[2];
  uint32_t sc[kPairs][2];
  auto load_pair = [&](int i, int r0, int r1) {
    const int q = 2 * i + team;
    if (q >= kQ) return;
#pragma unroll
    for (int g = 0; g < 2; ++g) {
      const size_t r = (size_t)max(g ? r1 : r0, 0);
      code[i][g] = __ldg(reinterpret_cast<const uint4*>(p.codes + r * (DV / 2) + part * (DV / 8)) + q);
      sc[i][g] = __ldg(reinterpret_cast<const uint32_t*>(p.scales + r * (DV / 32) + (part / 2) * (DV / 64)) + q);
    }
  };
  auto load_tail = [&](int r0, int r1) {
    const uint4* ts = reinterpret_cast<const uint4*>(p.tail + (size_t)max(team ? r1 : r0, 0) * 64) + part * 2;
    tail[0] = __ldg(ts);
    tail[1] = __ldg(ts + 1);
  };
  int r0 = c.row(p, x0), r1 = c.row(p, x0 + 8);
#pragma unroll
  for (int i = 0; i < kPairs; ++i) load_pair(i, r0, r1);
  load_tail(r0, r1);
  c.next(p, n_clusters);
  r0 = c.row(p, x0);                                   // the next tile's rows
  r1 = c.row(p, x0 + 8);
  const uint32_t lo = ((2 * part) ^ r8) * 16, hi = ((2 * part + 1) ^ r8) * 16;
  uint8_t* const out = k_sm + w4 * 2048 + r8 * 128;    // row group g: + 1024 g
  const uint32_t full0 = mapa_shared(smem_u32(&S.k_full[0]), 0);
  uint32_t tile_kc = 0;
  for (;;) {
    const bool more = c.u < p.n_units;
    const int n0 = r0, n1 = r1;
    c.next(p, n_clusters);
    r0 = c.row(p, x0);                                 // two tiles ahead
    r1 = c.row(p, x0 + 8);
#pragma unroll
    for (int i = 0; i < kPairs; ++i) {
      const int q = 2 * i + team;
      if (q >= kQ) continue;
      // Slots are freed in order: when the pair's second is free, so is its first.
      const uint32_t kc = tile_kc + 2 * q, s0 = kc % kKStages, s1 = (kc + 1) % kKStages;
      if (!mbar_wait_warp(&S.k_empty[s1], (((kc + 1) / kKStages) & 1u) ^ 1u, abort_flag)) return;
#pragma unroll 1
      for (int e = 0; e < 2; ++e) {
#pragma unroll
        for (int g = 0; g < 2; ++g) {
          store_codes(out + (e ? s1 : s0) * kPlane64 + g * 1024, lo, hi, code[i][g].x, code[i][g].y, sc[i][g] & 0xffffu);
          code[i][g].x = code[i][g].z;
          code[i][g].y = code[i][g].w;
          sc[i][g] >>= 16;
        }
      }
      if (more) load_pair(i, n0, n1);
      fence_proxy_async_smem();
      __syncwarp();
      // a team fills the slots that all eight warps fill for the tail: two arrivals each
      if (lane < 2) mbar_arrive_remote_n(full0 + (lane ? s1 : s0) * 8, 2);
    }
    const uint32_t kc = tile_kc + kLat, st = kc % kKStages;
    if (!mbar_wait_warp(&S.k_empty[st], ((kc / kKStages) & 1u) ^ 1u, abort_flag)) return;
    *reinterpret_cast<uint4*>(out + st * kPlane64 + team * 1024 + lo) = tail[0];
    *reinterpret_cast<uint4*>(out + st * kPlane64 + team * 1024 + hi) = tail[1];
    if (more) load_tail(n0, n1);
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) mbar_arrive_remote(full0 + st * 8);
    if (!more) break;
    tile_kc += NC;
  }
}

// Value loaders.  Team t does the tile's stages t, t + 2: this CTA's half of the columns of a
// value block, 64 rows.  A masked slot's row gets scale 0: zeros, whatever it holds.
template <int DV>
__device__ __forceinline__ void packed_values(const AttnParams& p, AttnBarriers& S, uint8_t* v_sm, int pw,
                                              uint32_t rank, int cluster_id, int n_clusters,
                                              volatile uint32_t* abort_flag) {
  using VS = VShape<DV>;
  constexpr int kVStages = Cfg<kPacked>::kVStages;
  constexpr int kPl = VS::kPlanes;                     // 64-column planes of a stage
  constexpr int kJobs = VS::kNpv;                      // per tile and team (two key halves x kNpv blocks, two teams)
  const int lane = (int)lane_id(), r8 = lane / 4, part = lane % 4, team = pw / 4, w4 = pw % 4;
  // Stage s is key half s / kNpv, block s % kNpv; team t's job i is stage 2 i + t.
  const int block = kJobs == 2 ? team : 0;
  const int x0 = (kJobs == 2 ? 0 : team * kHalfKeys) + w4 * 16 + r8;   // job i: + 64 i
  const int chunk = block * (VS::kN / 64) + (int)rank * kPl;           // of the stage's first plane
  TileCursor c;
  c.start(p, cluster_id, n_clusters);
  if (c.u >= p.n_units) return;
  uint4 code[kJobs][2];
  uint32_t sc[kJobs][2];
  int row[kJobs][2];
  auto rows = [&]() {
#pragma unroll
    for (int i = 0; i < kJobs; ++i)
#pragma unroll
      for (int g = 0; g < 2; ++g) row[i][g] = c.row(p, x0 + i * kHalfKeys + g * 8);
  };
  auto load = [&](int i, const int (&r)[2]) {
#pragma unroll
    for (int g = 0; g < 2; ++g) {
      const size_t at = (size_t)max(r[g], 0);
      const uint8_t* cs = p.codes + at * (DV / 2) + part * (DV / 8) + chunk * 8;
      const __nv_bfloat16* ss = p.scales + at * (DV / 32) + (part / 2) * (DV / 64) + chunk;
      if constexpr (kPl == 2) {
        code[i][g] = __ldg(reinterpret_cast<const uint4*>(cs));
        sc[i][g] = r[g] >= 0 ? __ldg(reinterpret_cast<const uint32_t*>(ss)) : 0u;
      } else {
        const uint2 v = __ldg(reinterpret_cast<const uint2*>(cs));
        code[i][g] = make_uint4(v.x, v.y, 0u, 0u);
        sc[i][g] = r[g] >= 0 ? __ldg(reinterpret_cast<const unsigned short*>(ss)) : 0u;
      }
    }
  };
  rows();
#pragma unroll
  for (int i = 0; i < kJobs; ++i) load(i, row[i]);
  c.next(p, n_clusters);
  rows();                                              // the next tile's
  const uint32_t lo = ((2 * part) ^ r8) * 16, hi = ((2 * part + 1) ^ r8) * 16;
  uint8_t* const out = v_sm + w4 * 2048 + r8 * 128;
  const uint32_t full0 = mapa_shared(smem_u32(&S.v_full[0]), 0);
  uint32_t st = (uint32_t)team, ph = 1;
  for (;;) {
    const bool more = c.u < p.n_units;
#pragma unroll
    for (int i = 0; i < kJobs; ++i) {
      if (!mbar_wait_warp(&S.v_empty[st], ph, abort_flag)) return;
#pragma unroll 1
      for (int pl = 0; pl < kPl; ++pl) {
#pragma unroll
        for (int g = 0; g < 2; ++g) {
          store_codes(out + st * VS::kStageBytes + pl * kPlane64 + g * 1024, lo, hi, code[i][g].x, code[i][g].y,
                      sc[i][g] & 0xffffu);
          code[i][g].x = code[i][g].z;
          code[i][g].y = code[i][g].w;
          sc[i][g] >>= 16;
        }
      }
      if (more) load(i, row[i]);
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive_remote(full0 + st * 8);
      st += 2;
      if (st >= kVStages) { st -= kVStages; ph ^= 1u; }
    }
    if (!more) break;
    c.next(p, n_clusters);
    rows();
  }
}

template <int NC, int DV, int MODE>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(Cfg<MODE>::kThreads, 1)
sparse_attn_kernel(const __grid_constant__ CUtensorMap tmap_q, const __grid_constant__ CUtensorMap tmap_kv,
                   const __grid_constant__ CUtensorMap tmap_kv_tile, const AttnParams p) {
  using VS = VShape<DV>;
  using C = Cfg<MODE>;
  static_assert(NC <= kMaxChunks, "d_qk");
  constexpr int kKStages = C::kKStages, kVStages = C::kVStages, kKWarp0 = C::kKWarp0, kKWarps = C::kKWarps;
  [[maybe_unused]] constexpr int kVWarp0 = C::kVWarp0, kVWarps = C::kVWarps, kKTeamWarps = C::kKTeamWarps;
  constexpr int kKTeamSlots = C::kKTeamSlots, kVWarpsPerSlot = C::kVWarpsPerSlot, kStageWarps = C::kStageWarps;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  AttnBarriers& S = *reinterpret_cast<AttnBarriers*>(smem_raw);
  // 1024-byte aligned operand area (the 128-byte swizzle is address based).
  const uint32_t raw_addr = smem_u32(smem_raw);
  const uint32_t area_off = ((raw_addr + sizeof(AttnBarriers) + 1023u) & ~1023u) - raw_addr;
  uint8_t* area = smem_raw + area_off;
  uint8_t* q_sm = area;                                             // NC planes
  uint8_t* k_sm = q_sm + NC * kPlane64;                             // kKStages planes
  uint8_t* v_sm = k_sm + kKStages * kPlane64;                       // kVStages x kPlanes planes
  uint8_t* p_sm = v_sm + kVStages * VS::kStageBytes;                // kPBufs x 2 planes
  int32_t* idx_sm = reinterpret_cast<int32_t*>(p_sm + kPBufs * 2 * kPlane64);  // 2 x kMaxIdx

  const uint32_t warp = warp_id();
  const uint32_t lane = lane_id();
  const uint32_t rank = cluster_ctarank();
  const bool leader = (rank == 0);
  const int cluster_id = blockIdx.x >> 1;
  const int n_clusters = gridDim.x >> 1;
  volatile uint32_t* abort_flag = &S.abort_flag;

  if (threadIdx.x == 0) {
    for (int i = 0; i < kMaxChunks; ++i) { mbar_init(&S.q_full[i], 1); mbar_init(&S.q_empty[i], 1); }
    for (int i = 0; i < kKStages; ++i) { mbar_init(&S.k_full[i], C::kKFillers); mbar_init(&S.k_empty[i], 1); }
    for (int i = 0; i < kVStages; ++i) { mbar_init(&S.v_full[i], C::kVFillers); mbar_init(&S.v_empty[i], 1); }
    for (int i = 0; i < kPBufs; ++i) {
      mbar_init(&S.p_full[i], 8);      // 4 softmax warps x 2 CTAs
      mbar_init(&S.p_empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&S.s_full[i], 1);
      mbar_init(&S.s_empty[i], 8);     // 4 softmax warps x 2 CTAs
      mbar_init(&S.idx_full[i], kStageWarps);
      mbar_init(&S.idx_empty[i], 4 + C::kIdxReaders);   // softmax warps + loader warps
    }
    mbar_init(&S.o_full, 1);
    mbar_init(&S.o_empty, 8);
    mbar_init(&S.final_s, 1);
    mbar_init(&S.final_pv, 1);
    mbar_init(&S.xbar[0], 2);
    mbar_init(&S.xbar[1], 2);
    S.abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == kMmaWarp) {
    tmem_alloc_pair(&S.tmem_base, kTmemCols);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();
  tc_fence_after();
  const uint32_t tmem_base = S.tmem_base;
  const uint16_t kBoth = 0x3;
  griddep_launch_dependents();
  griddep_wait();                                      // the previous kernel's writes are visible

  // Index staging (one warp of kStageWarps, number pw): each unit's selected positions
  // [j0*128, j1*128) go into buffer (unit ordinal % 2), one unit ahead, as the kv row to
  // load -- batch offset applied; padding and out-of-range entries gather row b*Lk
  // and are masked -- plus one validity ballot per 32 positions for the softmax
  // (kPacked: only the ballots).  Warp pw stages the 32-position words pw, pw + kStageWarps,
  // ...  A buffer is free again once the loaders and the softmax warps are done with
  // the unit two back.
  auto stage = [&](const Unit& V, uint32_t buf, int pw) {
    int32_t* dst = idx_sm + buf * kMaxIdx;
    uint32_t* vmask = S.valid_mask[buf];
    const int x_begin = V.j0 * kTileKeys, nwords = (V.j1 - V.j0) * (kTileKeys / 32);
    if (p.dense) {
      // Row t selects every position 0..t (in slot order); the bf16 loads need no
      // staged rows, only the validity words.  The leader also writes the
      // row's index list, and the first split its tail of -1 slots.
      int32_t* io = p.idx_out + (size_t)V.row * p.k;
      for (int w = pw; w < nwords; w += kStageWarps) {
        const int x = x_begin + w * 32 + (int)lane;
        const bool valid = x <= V.t && x < p.k;
        const uint32_t bal = __ballot_sync(0xffffffffu, valid);
        if (lane == 0) vmask[w] = bal;
        if (leader && x < p.k) io[x] = valid ? x : -1;
      }
      if (leader && V.split == 0) {
        const int nt_row = (min(p.k, V.t + 1) + kTileKeys - 1) / kTileKeys;
        for (int x = nt_row * kTileKeys + pw * 32 + (int)lane; x < p.k; x += kStageWarps * 32) io[x] = -1;
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&S.idx_full[buf]);
      return;
    }
    const int32_t* src = p.indices + (size_t)V.row * p.k;
    const int first = V.b * p.Lk, masked = p.zero_row ? p.zero_row : first;
    for (int w0 = pw; w0 < nwords; w0 += kStageWarps * kStageBatch) {
      int sidx[kStageBatch];
#pragma unroll
      for (int e = 0; e < kStageBatch; ++e) {
        const int w = w0 + e * kStageWarps, x = x_begin + w * 32 + (int)lane;
        sidx[e] = (w < nwords && x < p.k) ? __ldg(src + x) : -1;
      }
#pragma unroll
      for (int e = 0; e < kStageBatch; ++e) {
        const int w = w0 + e * kStageWarps;
        if (w >= nwords) break;                       // warp-uniform
        const bool valid = (sidx[e] >= 0) && (sidx[e] < p.Lk);
        if (MODE != kPacked) dst[w * 32 + (int)lane] = valid ? first + sidx[e] : masked;   // validity: the ballot below
        const uint32_t bal = __ballot_sync(0xffffffffu, valid);
        if (lane == 0) vmask[w] = bal;
      }
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(&S.idx_full[buf]);
  };

  if (warp >= 4) {
    if constexpr (C::kSplitRegs) regs_decrease<kRegsOther>();
    if (MODE == kPacked && warp >= kKWarp0) {
      // ------------------------------------------------------------------ converting loaders
      if constexpr (MODE == kPacked) {
        if (warp < kVWarp0)
          packed_keys<NC, DV>(p, S, k_sm, (int)warp - kKWarp0, rank, cluster_id, n_clusters, abort_flag);
        else
          packed_values<DV>(p, S, v_sm, (int)warp - kVWarp0, rank, cluster_id, n_clusters, abort_flag);
      }
    } else if (MODE == kPacked && warp > kPvWarp) {
      // ------------------------------------------------------------------ Q planes and index staging
      if constexpr (MODE == kPacked) {
        const int pw = (int)warp - (kPvWarp + 1);
        uint32_t ucount = 0;
        bool ok = true;
        if (pw == 0 && lane == 0) prefetch_tmap(&tmap_q);
        auto load_q = [&](const Unit& V) {               // planes pw, pw + kStageWarps, ...
          if (lane == 0) {
            const int qrow = V.row * p.H + (int)rank * 64;
            for (int c = pw; c < NC && ok; c += kStageWarps) {
              ok = mbar_wait(&S.q_empty[c], (ucount & 1u) ^ 1u, abort_flag);
              if (!ok) break;
              if (leader) mbar_arrive_expect_tx(&S.q_full[c], 2u * kPlane64);
              tma_load_2d_pair(q_sm + c * kPlane64, &tmap_q, mapa_shared(smem_u32(&S.q_full[c]), 0), c * 64, qrow);
            }
          }
          ok = __shfl_sync(0xffffffffu, ok, 0);
        };
        Unit U, Un;
        int u = next_unit<MODE>(p, cluster_id, n_clusters, U);
        if (u < p.n_units) {
          load_q(U);
          stage(U, 0, pw);
        }
        while (u < p.n_units && ok) {
          const int un = next_unit<MODE>(p, u + n_clusters, n_clusters, Un);
          if (ucount > 0) load_q(U);
          if (!ok) break;
          if (un < p.n_units) {
            const uint32_t nb = (ucount + 1) & 1u, nph = ((ucount + 1) >> 1) & 1u;
            // A whole unit's time to spare: sleep, so that the polls take no issue slots.
            for (int z = 0; z < 4096 && !mbar_test_wait(smem_u32(&S.idx_empty[nb]), nph ^ 1u); ++z) __nanosleep(500);
            ok = mbar_wait_warp(&S.idx_empty[nb], nph ^ 1u, abort_flag);
            if (!ok) break;
            stage(Un, nb, pw);
          }
          ++ucount;
          u = un;
          U = Un;
        }
      }
    } else if (warp >= kKWarp0 && warp < kVWarp0) {
      // ------------------------------------------------------------------ key loaders
      // Per unit: the Q planes (plane c from warp c % kKWarps), then for each tile
      // its NC key chunks (this CTA's 64 keys x 64 columns).  Chunk kc goes to
      // ring slot kc % kKStages; the team that owns that slot issues its 16
      // four-row gathers, groups g = part, part + kKTeamWarps, ...
      if constexpr (MODE != kPacked) {
      const int pw = (int)warp - kKWarp0;
      const uint32_t my_team = (uint32_t)(pw / kKTeamWarps);
      const int part = pw % kKTeamWarps;
      uint32_t ucount = 0, kc = 0;
      bool ok = true;
      if (pw == 0 && lane == 0) {
        prefetch_tmap(&tmap_q);
        prefetch_tmap(MODE == kWindow || p.dense ? &tmap_kv_tile : &tmap_kv);
      }
      Unit U;
      for (int u = next_unit<MODE>(p, cluster_id, n_clusters, U); u < p.n_units && ok;
           u = next_unit<MODE>(p, u + n_clusters, n_clusters, U)) {
        const uint32_t ib = ucount & 1u, uph = (ucount >> 1) & 1u;
        if (lane == 0) {
          const int qrow = U.row * p.H + (int)rank * 64;
          for (int c = pw; c < NC && ok; c += kKWarps) {
            ok = mbar_wait(&S.q_empty[c], (ucount & 1u) ^ 1u, abort_flag);
            if (!ok) break;
            if (leader) mbar_arrive_expect_tx(&S.q_full[c], 2u * kPlane64);
            tma_load_2d_pair(q_sm + c * kPlane64, &tmap_q, mapa_shared(smem_u32(&S.q_full[c]), 0), c * 64, qrow);
          }
        }
        ok = __shfl_sync(0xffffffffu, ok, 0);
        if (!ok) break;
        if (MODE != kWindow) ok = mbar_wait_warp(&S.idx_full[ib], uph, abort_flag);
        if (!ok) break;
        const int32_t* idx = idx_sm + ib * kMaxIdx;
        // The unit's chunks are kc_u .. kc_u + nk - 1; chunk x goes to slot x % kKStages.
        // The team visits only the chunks of its own slots (lo .. lo + kKTeamSlots - 1)
        // rather than stepping through all of them.
        const uint32_t kc_u = kc, nk = (uint32_t)(U.j1 - U.j0) * NC, lo = my_team * kKTeamSlots;
        uint32_t x = kc_u;
        {
          const uint32_t r = x % kKStages;
          if (r < lo) x += lo - r;
          else if (r >= lo + kKTeamSlots) x += kKStages - r + lo;
        }
        for (; x < kc_u + nk && ok; x += (x % kKStages + 1 < lo + kKTeamSlots) ? 1u : kKStages - kKTeamSlots + 1u) {
          const uint32_t st = x % kKStages, ph = (x / kKStages) & 1u;
          const int j = U.j0 + (int)((x - kc_u) / NC), c = (int)((x - kc_u) % NC);
          // Dense mode: one box per chunk from the team's first warp; the others
          // have nothing to load and must not wait either (a waiter that adds
          // nothing to a phase can fall two phases behind, where its parity test
          // would no longer see the phase it waits for).
          if (MODE == kSelected && p.dense && part != 0) continue;
          bool w_ok = true;
          if (lane == 0) {
            w_ok = mbar_wait(&S.k_empty[st], ph ^ 1u, abort_flag);
            if (w_ok && leader && part == 0) mbar_arrive_expect_tx(&S.k_full[st], 2u * kPlane64);
          }
          if (!__shfl_sync(0xffffffffu, w_ok, 0)) { ok = false; break; }
          const uint32_t full_l = mapa_shared(smem_u32(&S.k_full[st]), 0);
          if constexpr (MODE == kWindow) {
            if (lane < 16)
              window_load(p, U, j * kTileKeys + (int)rank * kHalfKeys, k_sm + st * kPlane64, &tmap_kv, &tmap_kv_tile,
                          full_l, c * 64, (int)lane);
            continue;
          }
          if (p.dense) {
            // keys 0..t are contiguous: this CTA's 64 rows of the tile in one box
            if (part == 0 && lane == 0)
              tma_load_2d_pair(k_sm + st * kPlane64, &tmap_kv_tile, full_l, c * 64,
                               U.b * p.Lk + j * kTileKeys + (int)rank * kHalfKeys);
            continue;
          }
          const int g = part + kKTeamWarps * (int)lane;            // 4-key group of this lane
          if (g < kHalfKeys / 4) {
            const int4 r4 = gather_rows4(idx, (j - U.j0) * kTileKeys + (int)rank * kHalfKeys + g * 4);
            tma_gather4_pair(k_sm + st * kPlane64 + g * 512, &tmap_kv, full_l, c * 64, r4.x, r4.y, r4.z, r4.w);
          }
        }
        kc = kc_u + nk;
        __syncwarp();
        if (MODE != kWindow && lane == 0) mbar_arrive(&S.idx_empty[ib]);
        ++ucount;
      }
      }
    } else if (warp >= kVWarp0) {
      // ------------------------------------------------------------------ value loaders
      // The value loaders also stage the indices, one unit ahead.
      // Value stages: per tile, 2 x kNpv stages of 64 keys (kh) x this CTA's kN/2
      // columns of value block h, i.e. all 128 keys of the tile across the two halves.
      if constexpr (MODE != kPacked) {
      const int pw = (int)warp - kVWarp0;
      const uint32_t my_slot = (uint32_t)(pw / kVWarpsPerSlot);
      const int part = pw % kVWarpsPerSlot;
      uint32_t ucount = 0, vc = 0;
      bool ok = true;
      Unit U, Un;
      int u = next_unit<MODE>(p, cluster_id, n_clusters, U);
      if (MODE != kWindow && u < p.n_units) stage(U, 0, pw);   // buffer 0 starts free
      while (u < p.n_units && ok) {
        const uint32_t ib = ucount & 1u, uph = (ucount >> 1) & 1u;
        const int un = next_unit<MODE>(p, u + n_clusters, n_clusters, Un);
        if (MODE != kWindow) {
          if (un < p.n_units) {
            const uint32_t nb = (ucount + 1) & 1u, nph = ((ucount + 1) >> 1) & 1u;
            ok = mbar_wait_warp(&S.idx_empty[nb], nph ^ 1u, abort_flag);
            if (!ok) break;
            stage(Un, nb, pw);
          }
          ok = mbar_wait_warp(&S.idx_full[ib], uph, abort_flag);
          if (!ok) break;
        }
        const int32_t* idx = idx_sm + ib * kMaxIdx;
        // The unit's value stages are vc_u .. vc_u + nv - 1 (per tile: key half kh,
        // then value block h); stage x goes to slot x % kVStages, and this warp visits
        // only its own slot's stages.
        constexpr uint32_t kPerTile = 2u * VS::kNpv;
        const uint32_t vc_u = vc, nv = (uint32_t)(U.j1 - U.j0) * kPerTile - (one_half<MODE>(U) ? VS::kNpv : 0);
        for (uint32_t x = vc_u + (my_slot + kVStages - vc_u % kVStages) % kVStages; x < vc_u + nv && ok;
             x += kVStages) {
          const uint32_t st = my_slot, ph = (x / kVStages) & 1u;
          const uint32_t rem = (x - vc_u) % kPerTile;
          const int j = U.j0 + (int)((x - vc_u) / kPerTile), kh = (int)(rem / VS::kNpv), h = (int)(rem % VS::kNpv);
          if (MODE == kSelected && p.dense && part != 0) continue;   // one issuing warp per slot (see the key loaders)
          bool w_ok = true;
          if (lane == 0) {
            w_ok = mbar_wait(&S.v_empty[st], ph ^ 1u, abort_flag);
            if (w_ok && leader && part == 0) mbar_arrive_expect_tx(&S.v_full[st], 2u * VS::kStageBytes);
          }
          if (!__shfl_sync(0xffffffffu, w_ok, 0)) { ok = false; break; }
          const uint32_t full_l = mapa_shared(smem_u32(&S.v_full[st]), 0);
          if constexpr (MODE == kWindow) {
            const int pl = (int)lane / 16;
            if (pl < VS::kPlanes)
              window_load(p, U, j * kTileKeys + kh * kHalfKeys, v_sm + st * VS::kStageBytes + pl * kPlane64, &tmap_kv,
                          &tmap_kv_tile, full_l, h * VS::kN + (int)rank * (VS::kN / 2) + pl * 64, (int)lane % 16);
            continue;
          }
          if (p.dense) {
            // 64 contiguous keys x this CTA's value columns: one box per plane
            if (part == 0 && lane < (uint32_t)VS::kPlanes) {
              const int col = h * VS::kN + (int)rank * (VS::kN / 2) + (int)lane * 64;
              tma_load_2d_pair(v_sm + st * VS::kStageBytes + lane * kPlane64, &tmap_kv_tile, full_l, col,
                               U.b * p.Lk + j * kTileKeys + kh * kHalfKeys);
            }
            continue;
          }
          const int g = part + kVWarpsPerSlot * (int)lane;
          if (g < 16 * VS::kPlanes) {
            const int pl = g / 16, kg = g % 16;
            const int4 r4 = gather_rows4(idx, (j - U.j0) * kTileKeys + kh * kHalfKeys + kg * 4);
            const int col = h * VS::kN + (int)rank * (VS::kN / 2) + pl * 64;
            tma_gather4_pair(v_sm + st * VS::kStageBytes + pl * kPlane64 + kg * 512, &tmap_kv, full_l, col,
                             r4.x, r4.y, r4.z, r4.w);
          }
        }
        vc = vc_u + nv;
        __syncwarp();
        if (MODE != kWindow && lane == 0) mbar_arrive(&S.idx_empty[ib]);
        ++ucount;
        u = un;
        U = Un;
      }
      }
    } else if (warp == kMmaWarp) {
      // ------------------------------------------------------------------ S issuer
      // S = Q K^T for each tile into TMEM buffer (tile ordinal % 2), one key chunk
      // (4 MMAs of K = 16) per ring stage.  S and P.V come from two threads so that
      // the single-thread issue rate bounds neither.
      if (leader && elect_one()) {
        constexpr uint32_t idesc_s = make_idesc(1, 1, 128, kTileKeys, 0, 0);       // bf16, K-major x K-major
        const uint64_t q_desc = make_smem_desc(smem_u32(q_sm), 16, 1024, LAYOUT_SW128);
        const uint64_t k_desc = make_smem_desc(smem_u32(k_sm), 16, 1024, LAYOUT_SW128);
        uint32_t ucount = 0, kc = 0, sc = 0;
        bool ok = true;
        Unit U;
        for (int u = next_unit<MODE>(p, cluster_id, n_clusters, U); u < p.n_units && ok;
             u = next_unit<MODE>(p, u + n_clusters, n_clusters, U)) {
          for (int j = U.j0; j < U.j1 && ok; ++j) {
            const uint32_t sb = sc & 1u;
            ok = mbar_wait(&S.s_empty[sb], ((sc >> 1) & 1u) ^ 1u, abort_flag, true);
            if (!ok) break;
            tc_fence_after();
            const uint32_t d = tmem_base + kTmemS + sb * kHalfKeys;
            for (int c = 0; c < NC; ++c) {
              if (j == U.j0 && !mbar_wait(&S.q_full[c], ucount & 1u, abort_flag)) { ok = false; break; }
              const uint32_t st = kc % kKStages, ph = (kc / kKStages) & 1u;
              if (!mbar_wait(&S.k_full[st], ph, abort_flag, MODE == kPacked)) { ok = false; break; }
              tc_fence_after();
              // descriptor start addresses advance 32 B (encoded 2) per K step of 16
              const uint64_t ad = q_desc + (uint64_t)(c * (kPlane64 >> 4));
              const uint64_t bd = k_desc + (uint64_t)(st * (kPlane64 >> 4));
              mma_bf16_ss_pair(d, ad + 0, bd + 0, idesc_s, c ? 1u : 0u);
              mma_bf16_ss_pair(d, ad + 2, bd + 2, idesc_s, 1u);
              mma_bf16_ss_pair(d, ad + 4, bd + 4, idesc_s, 1u);
              mma_bf16_ss_pair(d, ad + 6, bd + 6, idesc_s, 1u);
              mma_commit_pair_mc(&S.k_empty[st], kBoth);
              if (j == U.j1 - 1) mma_commit_pair_mc(&S.q_empty[c], kBoth);   // Q plane free for the next unit
              ++kc;
            }
            if (!ok) break;
            mma_commit_pair_mc(&S.s_full[sb], kBoth);
            ++sc;
          }
          ++ucount;
        }
        // Wait until every MMA this thread issued has completed before teardown.
        mma_commit(&S.final_s);
        mbar_wait(&S.final_s, 0, nullptr);
      }
    } else if (warp == kPvWarp) {
      // ------------------------------------------------------------------ P.V issuer
      // O += P V per tile: for each value stage (64 keys x kN value columns across
      // the pair), 4 MMAs of K = 16 keys reading P buffer (tile ordinal % 2).
      if (leader && elect_one()) {
        constexpr uint32_t idesc_pv = make_idesc(1, 1, 128, VS::kN, 0, 1);         // P K-major, V MN-major
        const uint64_t p_desc = make_smem_desc(smem_u32(p_sm), 16, 1024, LAYOUT_SW128);
        const uint64_t v_desc = make_smem_desc(smem_u32(v_sm), kPlane64, 1024, LAYOUT_SW128);
        uint32_t vc = 0, pc = 0, oc = 0;
        bool ok = true;
        Unit U;
        for (int u = next_unit<MODE>(p, cluster_id, n_clusters, U); u < p.n_units && ok;
             u = next_unit<MODE>(p, u + n_clusters, n_clusters, U)) {
          for (int j = U.j0; j < U.j1 && ok; ++j) {
            const bool first = (j == U.j0);
            ok = mbar_wait(&S.p_full[pc & 1u], (pc >> 1) & 1u, abort_flag, true);
            if (ok && first) ok = mbar_wait(&S.o_empty, (oc & 1u) ^ 1u, abort_flag, true);
            if (!ok) break;
            tc_fence_after();
            const int halves = j == U.j1 - 1 && one_half<MODE>(U) ? 1 : 2;
            for (int kh = 0; kh < halves && ok; ++kh) {
              for (int h = 0; h < VS::kNpv; ++h) {
                const uint32_t st = vc % kVStages, ph = (vc / kVStages) & 1u;
                if (!mbar_wait(&S.v_full[st], ph, abort_flag, MODE == kPacked)) { ok = false; break; }
                tc_fence_after();
                const uint32_t d = tmem_base + kTmemO + h * (VS::kN / 2);
                // P advances 32 B (encoded 2) and V 16 keys = 2048 B (encoded 128) per K step
                const uint64_t ad = p_desc + (uint64_t)(((pc & 1u) * 2 + kh) * (kPlane64 >> 4));
                const uint64_t bd = v_desc + (uint64_t)(st * (VS::kStageBytes >> 4));
                mma_bf16_ss_pair(d, ad + 0, bd + 0, idesc_pv, (first && kh == 0) ? 0u : 1u);
                mma_bf16_ss_pair(d, ad + 2, bd + 128, idesc_pv, 1u);
                mma_bf16_ss_pair(d, ad + 4, bd + 256, idesc_pv, 1u);
                mma_bf16_ss_pair(d, ad + 6, bd + 384, idesc_pv, 1u);
                mma_commit_pair_mc(&S.v_empty[st], kBoth);
                ++vc;
              }
            }
            if (!ok) break;
            mma_commit_pair_mc(&S.p_empty[pc & 1u], kBoth);
            if (j == U.j1 - 1) { mma_commit_pair_mc(&S.o_full, kBoth); ++oc; }
            ++pc;
          }
        }
        mma_commit(&S.final_pv);
        mbar_wait(&S.final_pv, 0, nullptr);
      }
    }
  } else {
    if constexpr (C::kSplitRegs) regs_increase<kRegsSoftmax>();
    // ------------------------------------------------------------------ softmax / epilogue
    const uint32_t l = warp * 32 + lane;          // TMEM lane = (key half, head)
    const uint32_t h = l & 63u;                   // head within this CTA
    const uint32_t half = l >> 6;                 // which 64 keys of the tile this lane holds
    const int head = (int)rank * 64 + (int)h;
    const uint32_t lane_addr = (warp * 32u) << 16;
    uint32_t ucount = 0, sc = 0, pc = 0, oc = 0, xph = 0;
    bool ok = true;
    for (int u = cluster_id; u < p.n_units && ok; u += n_clusters) {
      const Unit U = decode_unit<MODE>(p, u);
      if (U.j0 >= U.j1) {
        // An empty split: no keys.  Partial result is (O = 0, lse = -inf).
        if (p.splits > 1 && half == 0 && head < p.H) {
          const size_t prow = ((size_t)U.row * p.splits + U.split) * p.H + head;
          p.part_lse[prow] = -INFINITY;
          float4* o4 = reinterpret_cast<float4*>(p.part_o + prow * DV);
          for (int x = 0; x < DV / 4; ++x) o4[x] = make_float4(0.f, 0.f, 0.f, 0.f);
        }
        // A window row that sees nothing.
        if (MODE == kWindow && p.splits == 1 && half == 0 && head < p.H) {
          const size_t orow = (size_t)U.row * p.H + head;
          if (p.lse) p.lse[orow] = -INFINITY;
          uint4* o4 = reinterpret_cast<uint4*>(p.out + orow * DV);
          for (int x = 0; x < DV / 8; ++x) o4[x] = make_uint4(0u, 0u, 0u, 0u);
        }
        continue;
      }
      const uint32_t ib = ucount & 1u, uph = (ucount >> 1) & 1u;
      if (MODE != kWindow) ok = mbar_wait_warp(&S.idx_full[ib], uph, abort_flag);
      if (!ok) break;
      float m = -INFINITY, lsum = 0.f;
      for (int j = U.j0; j < U.j1 && ok; ++j) {
        const uint32_t sb = sc & 1u;
        ok = mbar_wait_warp(&S.s_full[sb], (sc >> 1) & 1u, abort_flag);
        if (!ok) break;
        tc_fence_after();
        // This lane's 64 logits, read from TMEM once.  Invalid entries (padding,
        // out-of-range) become -inf; whole groups are valid except in a row's last tile.
        const uint32_t s_addr = tmem_base + lane_addr + kTmemS + sb * kHalfKeys;
        uint32_t vmask0, vmask1;                      // warp-uniform
        if constexpr (MODE == kWindow) {
          const int n = U.n_valid - (j * kTileKeys + (int)half * kHalfKeys);
          vmask0 = n >= 32 ? 0xffffffffu : n <= 0 ? 0u : (1u << n) - 1u;
          vmask1 = n >= 64 ? 0xffffffffu : n <= 32 ? 0u : (1u << (n - 32)) - 1u;
        } else {
          const uint32_t* vm = &S.valid_mask[ib][((j - U.j0) * kTileKeys + (int)half * kHalfKeys) / 32];
          vmask0 = vm[0];
          vmask1 = vm[1];
        }
        uint32_t v[64];
        tmem_ld32(s_addr, *reinterpret_cast<uint32_t(*)[32]>(&v[0]));
        tmem_ld32(s_addr + 32, *reinterpret_cast<uint32_t(*)[32]>(&v[32]));
        tmem_ld_wait();
        if ((vmask0 & vmask1) != 0xffffffffu) {
#pragma unroll
          for (int c = 0; c < 64; ++c)
            if (!((((c < 32) ? vmask0 : vmask1) >> (c & 31)) & 1u)) v[c] = __float_as_uint(-INFINITY);
        }
        float smax = -INFINITY;                       // maximum of the raw logits (scale > 0)
#pragma unroll
        for (int c = 0; c < 64; ++c) smax = fmaxf(smax, __uint_as_float(v[c]));
        float tmax = smax * p.scale_log2;
        const uint32_t rb = sc & 1u;
        S.red_max[rb][l] = tmax;
        ok = warps_rendezvous(&S.xbar[warp & 1u], xph, abort_flag);
        if (!ok) break;
        tmax = fmaxf(tmax, S.red_max[rb][l ^ 64u]);
        const float m_new = fmaxf(m, tmax);
        const bool first = (j == U.j0);
        const bool need = first || (m_new > m + kRescaleThreshold);
        const float m_ref = need ? m_new : m;
        const float m_use = (m_ref == -INFINITY) ? 0.f : m_ref;
        // P buffer pc % 2 is free once the P.V two tiles back is done.
        const uint32_t pbuf = pc & 1u;
        ok = mbar_wait_warp(&S.p_empty[pbuf], ((pc >> 1) & 1u) ^ 1u, abort_flag);
        if (!ok) break;
        tc_fence_after();
        if (!first && __any_sync(0xffffffffu, need)) {
          // Rescaling O needs the previous tile's P.V to be complete.
          ok = mbar_wait_warp(&S.p_empty[pbuf ^ 1u], ((pc - 1u) >> 1) & 1u, abort_flag);
          if (!ok) break;
          tc_fence_after();
          const float alpha = need ? exp2f(m - m_new) : 1.f;
          for (int c0 = 0; c0 < VS::kNpv * (VS::kN / 2); c0 += 16) {
            uint32_t ov[16];
            tmem_ld16(tmem_base + lane_addr + kTmemO + c0, ov);
            tmem_ld_wait();
#pragma unroll
            for (int e = 0; e < 16; ++e) ov[e] = __float_as_uint(__uint_as_float(ov[e]) * alpha);
            tmem_st16(tmem_base + lane_addr + kTmemO + c0, ov);
          }
          tmem_st_wait();
          if (need) lsum *= alpha;
        }
        if (need) m = m_new;
        // Probabilities 2^(z*scale*log2e - m), packed to bf16 straight into P (row h of
        // this lane's key-half plane, 128-byte swizzle); the row sum is kept in fp32.  The
        // product with the bf16 values takes bf16 (both operands of an MMA have one type):
        // every probability is off by at most 2^-8 of itself, which makes the output's
        // error 2.1e-3 of its size where its own rounding alone leaves 1.7e-3.
        uint8_t* prow = p_sm + (pbuf * 2 + half) * kPlane64 + (h >> 3) * 1024 + (h & 7) * 128;
        const float2 scl = make_float2(p.scale_log2, p.scale_log2);
        const float2 nm = make_float2(-m_use, -m_use);
        float2 sum2 = make_float2(0.f, 0.f);
#pragma unroll
        for (int q = 0; q < 8; ++q) {                   // 16-byte chunk q: keys 8q .. 8q+7
          uint32_t w4[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int c0 = q * 8 + 2 * e;
            const float2 x = ffma2(make_float2(__uint_as_float(v[c0]), __uint_as_float(v[c0 + 1])), scl, nm);
            const float2 pr = make_float2(ex2_approx(x.x), ex2_approx(x.y));
            sum2 = fadd2(sum2, pr);
            const __nv_bfloat162 b2 = __floats2bfloat162_rn(pr.x, pr.y);
            w4[e] = *reinterpret_cast<const uint32_t*>(&b2);
          }
          *reinterpret_cast<uint4*>(prow + ((q ^ (h & 7)) * 16)) = make_uint4(w4[0], w4[1], w4[2], w4[3]);
        }
        const float psum = sum2.x + sum2.y;
        lsum += psum;
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_remote(mapa_shared(smem_u32(&S.s_empty[sb]), 0));
        ++sc;
        fence_proxy_async_smem();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_remote(mapa_shared(smem_u32(&S.p_full[pbuf]), 0));
        ++pc;
      }
      if (!ok) break;
      __syncwarp();
      if (MODE != kWindow && lane == 0) mbar_arrive(&S.idx_empty[ib]);
      ++ucount;
      // ---- epilogue of the unit
      ok = mbar_wait_warp(&S.o_full, oc & 1u, abort_flag);
      ++oc;
      if (!ok) break;
      tc_fence_after();
      S.red_sum[l] = lsum;
      ok = warps_rendezvous(&S.xbar[warp & 1u], xph, abort_flag);
      if (!ok) break;
      const float total = lsum + S.red_sum[l ^ 64u];
      ok = warps_rendezvous(&S.xbar[warp & 1u], xph, abort_flag);   // red_sum may be rewritten next unit
      if (!ok) break;
      // A NaN logit (or one of +inf, minus the maximum) is in the sum, though a maximum passes
      // it over: out and lse are NaN then, and the merge of a split row carries it on.
      const float inv = total > 0.f ? 1.f / total : total;
      const float lse_v = total > 0.f ? (m + log2f(total)) * kLn2 : total == 0.f ? -INFINITY : total;
      const bool write = head < p.H;
      for (int hi = 0; hi < VS::kNpv; ++hi) {
        for (int c0 = 0; c0 < VS::kN / 2; c0 += 32) {
          uint32_t ov[32];
          tmem_ld32(tmem_base + lane_addr + kTmemO + hi * (VS::kN / 2) + c0, ov);
          tmem_ld_wait();
          const int dv0 = hi * VS::kN + (int)half * (VS::kN / 2) + c0;
          if (!write) continue;
          if (p.splits == 1) {
            __nv_bfloat16* dst = p.out + ((size_t)U.row * p.H + head) * DV + dv0;
#pragma unroll
            for (int e = 0; e < 32; e += 8) {
              uint4 w;
              w.x = pack_bf16(__uint_as_float(ov[e + 0]) * inv, __uint_as_float(ov[e + 1]) * inv);
              w.y = pack_bf16(__uint_as_float(ov[e + 2]) * inv, __uint_as_float(ov[e + 3]) * inv);
              w.z = pack_bf16(__uint_as_float(ov[e + 4]) * inv, __uint_as_float(ov[e + 5]) * inv);
              w.w = pack_bf16(__uint_as_float(ov[e + 6]) * inv, __uint_as_float(ov[e + 7]) * inv);
              *reinterpret_cast<uint4*>(dst + e) = w;
            }
          } else {
            float* dst = p.part_o + (((size_t)U.row * p.splits + U.split) * p.H + head) * DV + dv0;
#pragma unroll
            for (int e = 0; e < 32; e += 4)
              *reinterpret_cast<float4*>(dst + e) =
                  make_float4(__uint_as_float(ov[e]) * inv, __uint_as_float(ov[e + 1]) * inv,
                              __uint_as_float(ov[e + 2]) * inv, __uint_as_float(ov[e + 3]) * inv);
          }
        }
      }
      if (write && half == 0) {
        if (p.splits == 1) {
          if (p.lse) p.lse[(size_t)U.row * p.H + head] = lse_v;
        } else {
          p.part_lse[((size_t)U.row * p.splits + U.split) * p.H + head] = lse_v;
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_remote(mapa_shared(smem_u32(&S.o_empty), 0));
    }
  }

  tc_fence_before();
  __syncthreads();
  cluster_sync();
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc_pair(tmem_base, kTmemCols);
  }
}

// Merge split-k partials: lse = log sum_i exp(lse_i); out = sum_i exp(lse_i - lse) o_i.
// A split whose lse is NaN makes the row's out and lse NaN.
template <int DV>
__global__ void __launch_bounds__(128) attn_combine_kernel(const AttnParams p) {
  griddep_launch_dependents();
  griddep_wait();                                      // the partials are complete
  const int warps = blockDim.x / 32;
  const int gw = blockIdx.x * warps + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  const int n = p.B * p.Lq * p.H;
  if (gw >= n) return;
  const int row = gw / p.H, head = gw % p.H;
  float mx = -INFINITY;
  bool any = false;                                    // a split saw something
  for (int sp = 0; sp < p.splits; ++sp) {
    const float l = p.part_lse[((size_t)row * p.splits + sp) * p.H + head];
    mx = fmaxf(mx, l);
    any = any || l != -INFINITY;
  }
  float wsum = 0.f;
  float acc[DV / 32];
#pragma unroll
  for (int e = 0; e < DV / 32; ++e) acc[e] = 0.f;
  if (any) {
    for (int sp = 0; sp < p.splits; ++sp) {
      const size_t prow = ((size_t)row * p.splits + sp) * p.H + head;
      const float wgt = expf(p.part_lse[prow] - mx);
      wsum += wgt;
      const float* src = p.part_o + prow * DV;
#pragma unroll
      for (int e = 0; e < DV / 32; ++e) acc[e] = fmaf(wgt, src[e * 32 + lane], acc[e]);
    }
  }
  const float inv = wsum > 0.f ? 1.f / wsum : wsum;
  __nv_bfloat16* dst = p.out + ((size_t)row * p.H + head) * DV;
#pragma unroll
  for (int e = 0; e < DV / 32; ++e) dst[e * 32 + lane] = __float2bfloat16_rn(acc[e] * inv);
  if (lane == 0 && p.lse) p.lse[(size_t)row * p.H + head] = wsum > 0.f ? mx + logf(wsum) : wsum == 0.f ? -INFINITY : wsum;
}

template <int NC, int DV, int MODE>
cudaError_t launch_t(const AttnParams& p, const CUtensorMap& tq, const CUtensorMap& tkv,
                     const CUtensorMap& tkv_tile, int grid_clusters, cudaStream_t stream) {
  using C = Cfg<MODE>;
  constexpr size_t smem = sizeof(AttnBarriers) + 1024              // barriers + alignment slack
                          + (size_t)NC * kPlane64                  // Q
                          + (size_t)C::kKStages * kPlane64         // K ring
                          + (size_t)C::kVStages * VShape<DV>::kStageBytes   // V ring
                          + (size_t)kPBufs * 2 * kPlane64          // P buffers (keys 0-63, 64-127 each)
                          + (MODE == kSelected ? 2 * (size_t)kMaxIdx * sizeof(int32_t) : 0);   // staged indices, two units
  static_assert(smem <= 232448, "shared memory of one CTA");
  auto kern = sparse_attn_kernel<NC, DV, MODE>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  // The register split must fit in what the CTA launches with, or the increase
  // would wait forever: refuse to launch a build where it does not.  (A property of
  // the binary: asked for once.)
  if constexpr (C::kSplitRegs) {
    static std::atomic<bool> fits{false};
    if (!fits.load(std::memory_order_relaxed)) {
      cudaFuncAttributes fa;
      e = cudaFuncGetAttributes(&fa, kern);
      if (e != cudaSuccess) return e;
      if ((uint32_t)fa.numRegs < kRegsLaunch) return cudaErrorInvalidConfiguration;
      fits.store(true, std::memory_order_relaxed);
    }
  }
  return launch_pdl(kern, dim3(grid_clusters * 2), dim3(C::kThreads), smem, stream, tq, tkv, tkv_tile, p);
}

}  // namespace

cudaError_t launch_sparse_attn(const AttnParams& p, int d_qk, int d_v, const CUtensorMap& tq,
                               const CUtensorMap& tkv, const CUtensorMap& tkv_tile, int grid_clusters,
                               cudaStream_t stream) {
  const bool mla = d_qk == 576 && d_v == 512;
  if (!mla && !(d_qk == 192 && d_v == 128)) return cudaErrorInvalidValue;
  if (p.codes)
    return mla ? launch_t<9, 512, kPacked>(p, tq, tkv, tkv_tile, grid_clusters, stream)
               : launch_t<3, 128, kPacked>(p, tq, tkv, tkv_tile, grid_clusters, stream);
  if (p.window)
    return mla ? launch_t<9, 512, kWindow>(p, tq, tkv, tkv_tile, grid_clusters, stream)
               : launch_t<3, 128, kWindow>(p, tq, tkv, tkv_tile, grid_clusters, stream);
  return mla ? launch_t<9, 512, kSelected>(p, tq, tkv, tkv_tile, grid_clusters, stream)
             : launch_t<3, 128, kSelected>(p, tq, tkv, tkv_tile, grid_clusters, stream);
}

cudaError_t launch_attn_combine(const AttnParams& p, int d_v, cudaStream_t stream) {
  const int n = p.B * p.Lq * p.H;
  const int grid = (n + 3) / 4;
  if (d_v == 512) return launch_pdl(attn_combine_kernel<512>, dim3(grid), dim3(128), 0, stream, p);
  if (d_v == 128) return launch_pdl(attn_combine_kernel<128>, dim3(grid), dim3(128), 0, stream, p);
  return cudaErrorInvalidValue;
}

cudaError_t read_attn_error(uint32_t* value, bool clear) { return read_unit_error(value, clear); }

}  // namespace dsa
