// Attention of a chunk of new tokens (more packed query rows than the token kernel takes)
// over a paged cache, on the tensor cores.
//
// An item is 256 packed rows (token, head of the group) of one sequence and kv head, as two
// slots of 128 rows that share every K and V tile.  With 2 * 128 rows a tile of 128 keys costs
// 4 * 128 * 128 * d multiply-adds, 2048 cycles of the tensor pipe at d = 128, against about 1400
// cycles for its K and V from HBM and less from L2: the products bound it, so everything
// else is arranged to keep them fed.  One CTA an SM, 16 warps (20 with an e4m3 cache):
//   warp 0          issues tcgen05.mma: S_w = Q_w K^T into TMEM, then O_w += P_w V with P_w read
//                   from TMEM over the columns of S_w; the order PV0, S0, PV1, S1 lets each slot's
//                   softmax run under the other slot's products;
//   warp 3          walks the CTA's run and publishes its parts, one item or piece of an item
//                   each, in shared memory for the other roles (which keeps the walk's
//                   state out of their registers: spilled there it cost more than half the time);
//   warps 1 and 2   look through the V tiles (by TMA) whose keys not every row sees: rows that nobody
//                   sees become zeros, values that are not finite are cleared (fdma_paged.cuh);
//                   the loads stay ahead meanwhile; with an e4m3 cache they bring its codes (a box
//                   for 16 keys) and its scale bytes instead, and the converting warps look;
//   warps 4..7,     softmax of slot 0 and slot 1, one thread a row: masked only in tiles that some
//   warps 8..11     row of the warp sees in part, exponentiated with a running maximum that is
//                   raised only when it grows by 2^8 or more;
//   warps 12..      bring Q, K and V into 128-byte-swizzled tiles: a ring of five bf16 tiles by TMA, a
//                   box a page, or by cp.async where TMA cannot address the cache's layout or a page
//                   is not there; or turn an e4m3 cache's codes into a ring of four tiles: multiplied
//                   by their scale and stored as bf16 (exact down to bf16's least step, 2^-133).
// The line of all items' tiles is cut into one run a CTA (fdma_paged.cuh), so a causal chunk or
// a ragged batch keeps every SM busy to the end; the ring and the barriers run on across items.
//
// 2048 tokens over 16384 keys, 16 heads on 4 kv heads of 128, bf16: 171 us, 1.51 PFLOP/s, from a captured graph (184 us, 1.40
// PFLOP/s, a call).  A slot's softmax
// waits for its S and its next S for its P, about 3300 cycles a tile with the other slot's
// products in between.  e4m3 (333 to 1024 tokens of two sequences over 4097 to 8192 keys, 32 heads): 127 us;
// the conversion, 1300 cycles an item, and the longer softmax share the issue slots.
#include "fdma_paged.cuh"

namespace fdma {
namespace {

constexpr int kChunkRows = kChunkItemRows;
constexpr int kKeyTile = 128;
constexpr int kRingTiles = 5;  // K and V tiles in shared memory (four, and kRaw raw ones, with e4m3)
constexpr int kRaw = 2;     // (four, and a ring of three, took 133 instead of 130 us below)
constexpr int kScales = 2;  // tiles' scale bytes
constexpr int kParts = 4;  // published parts
constexpr int kLooks = 4;  // V tiles to be looked through: an entry is free again when the ring has gone round
// Loading warps and the division of the registers (setmaxnreg).  An e4m3 cache has eight loading warps,
// because the conversion of its tiles to bf16 bounds it, and the softmax keeps less in registers for
// it: the e4m3 case above took 199 us with four such warps (and each row's scores in registers), 131 with eight.
template <bool FP8>
struct ChunkRoles {
  static constexpr int kLoadWarps = FP8 ? 8 : 4;
  static constexpr int kThreads = 384 + 32 * kLoadWarps;
  static constexpr uint32_t kRegsMma = 64, kRegsLoad = FP8 ? 96 : 80, kRegsSoft = FP8 ? 112 : 184;
  static constexpr int kLaunchRegs = FP8 ? 96 : 128;
  static_assert(kRegsMma + kRegsLoad * (kLoadWarps / 4) + 2 * kRegsSoft == kLaunchRegs * (kThreads / 128),
                "the registers of the launch");
};
constexpr uint64_t kIdleWaitNs = 300ull * kWaitLimitNs;
constexpr float kNInf = -__builtin_huge_valf();
constexpr float kRaise = 8.f;  // log2 units: P stays at most 2^8 between raises of the maximum

enum ChunkBar : int {
  cFull = 0,             // + ring slot: the loading warps
  cEmpty = kRingTiles,   // + ring slot: the products that read it are done
  cQFull = 2 * kRingTiles,  // the part's Q is in shared memory
  cQEmpty,                  // the part's last S product is done
  cSFull,                // + slot
  cPReady = cSFull + 2,  // + 2 * slot + key half
  cOFinal = cPReady + 4,  // + slot: the item's last PV is done
  cOFree = cOFinal + 2,   // + slot: the softmax threads have read O
  cPart = cOFree + 2,     // + part slot: the part is published
  cPartFree = cPart + kParts,  // + part slot: every reader is done with it
  cLook = cPartFree + kParts,  // + entry: a V tile to be looked through has landed
  cDrain = cLook + kLooks,
  cRaw,  // + place: an e4m3 item's codes are in shared memory
  cRawFree = cRaw + kRaw,  // + place: they have been converted
  cScale = cRawFree + kRaw,  // + place: the scale bytes of a tile's K and V rows
  cScaleFree = cScale + kScales,
  kChunkBars = cScaleFree + kScales
};

// Byte offset of 16-byte chunk c of row r in a K-major tile of 64-column blocks, 128-byte swizzle.
__device__ __forceinline__ uint32_t tile_off(int r, int c) {
  return (c >> 3) * 16384 + r * 128 + (((c & 7) ^ (r & 7)) << 4);
}

// A CTA's part of one item: its tiles t0 .. t0 + n - 1.
struct Part {
  int n;      // 0: the run is over
  int whole;  // the item's tiles are all here: the result is final
  int slot;   // else: where its sums go in the workspace
  int slots;  // row slots in use
  int t0, sink_tiles, main0;
  int lo, hi, sink_hi;
  int b, g, row0;  // row0: first packed row
  int all_lo, all_hi;  // keys j < all_hi with j >= all_lo or j < sinks are seen by every row
  int q0, nq, pos0, klen;
  int odd;  // set by the loads: values that are not finite were cleared
};
// First key of the k-th tile of a part.
struct PartTiles {
  int t0, sink_tiles, skip;
  __device__ __forceinline__ explicit PartTiles(const Part& s)
      : t0(s.t0), sink_tiles(s.sink_tiles), skip(s.main0 - s.sink_tiles) {}
  __device__ __forceinline__ int key0(int k) const {
    const int t = t0 + k;
    return (t < sink_tiles ? t : t + skip) * kKeyTile;
  }
};

// True in one lane of a converged warp, the same one every time.
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
  return r != 0;
}

struct Look {
  int slot;  // of the ring; -1: the run is over
  int j0, part;
};

__device__ __forceinline__ SeenKeys part_seen(const Part& s, int sinks) {
  return SeenKeys{s.lo, s.hi, s.sink_hi, s.all_lo, s.all_hi, sinks};
}

// A place in a ring of N tiles and the parity of its current fill.
template <int N>
struct RingPos {
  int slot = 0;
  uint32_t phase = 0;
  __device__ __forceinline__ void step() {
    if (++slot == N) {
      slot = 0;
      phase ^= 1;
    }
  }
};

template <int D, bool FP8>
struct ChunkSmem {
  static constexpr int kTile = 128 * D * 2;
  static constexpr int kRing = FP8 ? 4 : kRingTiles;
  static constexpr int kOffRing = 2 * kTile;
  static constexpr int kOffRaw = kOffRing + kRing * kTile;  // e4m3: [kRaw] items' rows of d codes
  static constexpr int kOffScale = kOffRaw + (FP8 ? kRaw * (kTile / 2) : 0);  // [kScales][K, V][128]
  static constexpr int kOffAbsent = kOffScale + (FP8 ? kScales * 256 : 0);    // [kRaw]: groups of 16 rows that are not there
  static constexpr int kOffBar = kOffAbsent + (FP8 ? kRaw * 4 : 0);
  static constexpr int kOffMisc = kOffBar + kChunkBars * 8;
  static constexpr int kOffParts = kOffMisc + 16;
  static constexpr int kOffLooks = kOffParts + kParts * static_cast<int>(sizeof(Part));
  static constexpr int kOffPlan = (kOffLooks + kLooks * static_cast<int>(sizeof(Look)) + 7) / 8 * 8;
  static constexpr int kTotal = kOffPlan + static_cast<int>(sizeof(PlanSmem));
  static_assert(kTotal <= 232448, "shared memory of one CTA");
};

template <int D, bool FP8>
__global__ void __launch_bounds__(ChunkRoles<FP8>::kThreads, 1)
    paged_chunk_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                       const __grid_constant__ PagedParams p) {
  using L = ChunkSmem<D, FP8>;
  using Roles = ChunkRoles<FP8>;
  constexpr int LT = 32 * Roles::kLoadWarps;  // loading threads
  using Ring = RingPos<L::kRing>;
  constexpr int ROWS = kChunkRows;
  constexpr uint32_t IDESC_S = idesc_bf16(128, 128, false, false);
  constexpr uint32_t IDESC_O = idesc_bf16(128, D, false, true);
  extern __shared__ __align__(1024) uint8_t smem[];
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L::kOffBar);
  uint32_t* misc = reinterpret_cast<uint32_t*>(smem + L::kOffMisc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(misc + 1);
  PlanSmem* plan = reinterpret_cast<PlanSmem*>(smem + L::kOffPlan);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  if ((smem_u32(smem) & 1023u) != 0) {
    if (tid == 0) atomicCAS(p.err, 0, kDevErrAlign);
    return;
  }
  Cursor<ROWS, kKeyTile> c;
  int quota;
  const bool any = plan_run<ROWS, kKeyTile, Roles::kThreads>(p, plan, c, quota);
  if (tid == 0) p.desc[blockIdx.x] = make_int4(0, 0, 0, 0);
  write_empty_blocks<ROWS>(p);
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (!any) return;

  if (tid == 0) {
    for (int i = 0; i < kChunkBars; ++i) mbar_init(&bars[i], 1);
    for (int i = 0; i < kRingTiles; ++i) mbar_init(&bars[cFull + i], Roles::kLoadWarps);
    mbar_init(&bars[cQFull], Roles::kLoadWarps);
    for (int i = 0; i < 4; ++i) mbar_init(&bars[cPReady + i], 128);
    for (int i = 0; i < 2; ++i) mbar_init(&bars[cOFree + i], 128);
    for (int i = 0; i < kRaw; ++i) mbar_init(&bars[cRawFree + i], Roles::kLoadWarps);
    for (int i = 0; i < kScales; ++i) mbar_init(&bars[cScaleFree + i], Roles::kLoadWarps);
    for (int i = 0; i < kParts; ++i) mbar_init(&bars[cPartFree + i], LT + 1 + 256 + (FP8 ? 2 : 0));
    misc[1] = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(misc, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tbase = misc[0];
  uint8_t* sQ = smem;
  uint8_t* sR = smem + L::kOffRing;
  auto wait = [&](int bar, uint32_t parity) { return mbar_wait(&bars[bar], parity, p.err, kDevErrTimeout, abort_flag); };

  // For whole warps that go on to warp-wide instructions: every lane gets the same answer, whichever of them
  // saw the time-out, so that none waits for lanes that have left (1 % of the time of a call).
  auto wait_all = [&](int bar, uint32_t parity) { return __all_sync(0xffffffffu, wait(bar, parity)) != 0; };
  // For the roles that have nothing to do for most of a run, however long it is; a time-out of
  // another role ends these waits too.
  auto idle_wait = [&](int bar, uint32_t parity) {
    return mbar_wait(&bars[bar], parity, p.err, kDevErrTimeout, abort_flag, kIdleWaitNs);
  };

  Part* parts = reinterpret_cast<Part*>(smem + L::kOffParts);
  Look* look_at = reinterpret_cast<Look*>(smem + L::kOffLooks);
  // The idx-th part of the run; false on a time-out.
  auto part_ready = [&](int idx) { return wait(cPart + idx % kParts, (idx / kParts) & 1); };
  auto part_ready_all = [&](int idx) { return wait_all(cPart + idx % kParts, (idx / kParts) & 1); };
  auto part_done = [&](int idx) { mbar_arrive(&bars[cPartFree + idx % kParts]); };

  if (warp >= 12) {
    // ------------------------------------------------------------------ loads
    // Items (K_0, V_0, K_1, V_1, ... of every part in turn) are brought ahead of the products as far
    // as the ring goes, across parts.
    regs_decrease<Roles::kRegsLoad>();
    const int lt = tid - 384;
    const int pmask = (1 << p.c.page_shift) - 1;
    Ring at;     // the place of the next item
    int it = 0;  // items issued
    bool ok = true;
    // every thread of the warp has stored its part of what `bar` announces
    auto announce = [&](int bar) {
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars[bar]);
    };
    auto slot_free = [&](int item) { return item < L::kRing || wait_all(cEmpty + at.slot, at.phase ^ 1); };
    // A thread has one 16-byte column (of the cache's row) of NP rows r0 + i * RPP; with an e4m3 cache these
    // are of the warp's group of 16 keys.
    constexpr int CPR = FP8 ? D / 16 : D / 8, RPP = (FP8 ? 32 : LT) / CPR, NP = (FP8 ? 16 : 128) / RPP;
    constexpr int NB = NP < 4 ? NP : 4;
    static_assert(!FP8 || Roles::kLoadWarps == 8, "a warp for each 16 of a tile's 128 keys");
    const int chunk = lt % CPR, r0 = FP8 ? (warp - 12) * 16 + lane / CPR : lt / CPR;
    const uint32_t cb = chunk * 16 < p.c.d * (FP8 ? 1 : 2) ? 16u : 0u;
    // e4m3: this thread's first piece of the item at place 0; piece i lies i * 512 on
    const uint32_t raw = smem_u32(smem) + L::kOffRaw + (warp - 12) * 16 * D + lane * 16;
    int looks = 0;  // bf16: V tiles given to the looking warps
    // (Rolled loops and one copy of each step: with the steps unrolled and inlined twice the roles'
    // code fell out of the instruction cache and everything ran at half speed.)
    for (int idx = 0; ok; ++idx) {
      if (!(ok = part_ready_all(idx))) break;
      Part& s = parts[idx % kParts];
      // (copies: what lies in shared memory is read again after every barrier)
      const int n = s.n, b = s.b, g_kv = s.g, lo = s.lo, hi = s.hi, sink_hi = s.sink_hi, all_lo = s.all_lo, all_hi = s.all_hi;
      const PartTiles tiles(s);
      // bf16: lanes 0..7 of every warp look up the pages of a tile's eight groups of 16 keys, one tile
      // ahead of their use; none where no row sees a key of the group (of its box).
      const int unit = max(p.box, 16);
      auto look_up = [&](int k) {
        int entry = kNoKeys;
        if (!FP8 && lane < 8 && k < n) {
          const int j = tiles.key0(k) + lane * 16, jb = j & -unit;
          if (jb < sink_hi || (jb < hi && jb + unit > lo)) entry = table_entry(p, b, j);
        }
        return entry;
      };
      int pg = -1, pg_next = look_up(0);
      bool missing = false;  // a page that is needed is not there
      unsigned boxes = 0;
      bool mine_box = false;
#pragma unroll 1
      for (int i2 = 0; i2 < 2 * n; ++i2) {
        const bool is_v = i2 & 1;
        const int j0 = tiles.key0(i2 >> 1);
        // V of keys that not every row sees is looked through.  (K needs no care: scores of unseen keys are
        // replaced, whatever they are.)
        const bool look = is_v && !(j0 >= all_lo && j0 + 128 <= all_hi);
        if (!FP8) {
          if (!is_v) {
            const int entry = pg_next;
            pg = checked_page(p, entry);
            missing = __any_sync(0xffffffffu, entry != kNoKeys && pg < 0);
            pg_next = look_up((i2 >> 1) + 1);
            // lane g brings the page of its group of 16 keys, if that group begins a box; the boxes are dealt
            // out over the four warps (a warp's boxes go one after the other)
            const bool begins = lane < 8 && ((lane * 16) & (unit - 1)) == 0 && pg >= 0;
            boxes = __ballot_sync(0xffffffffu, begins);
            mine_box = begins && ((lane * 16 / unit) & 3) == warp - 12;
          }
          if (!(ok = slot_free(it))) break;
          const int bar = cFull + at.slot;
          uint8_t* to = sR + at.slot * L::kTile;
          if (p.box > 0 && !missing) {
            uint64_t* to_bar = &bars[look ? cLook + looks % kLooks : bar];
            if (lane == 0) {
              if (warp == 12) {
                if (look) look_at[looks % kLooks] = Look{at.slot, j0, idx};
                mbar_arrive_expect_tx(to_bar, __popc(boxes) * p.box * (2 * D));
              } else if (!look) {
                mbar_arrive(to_bar);
              }
            }
            if (mine_box) {
              const CUtensorMap* tm = is_v ? &tmV : &tmK;
#pragma unroll
              for (int c = 0; c < D / 64; ++c)
                tma_load_4d(to + c * 16384 + lane * 2048, tm, to_bar, c * 64, (j0 + lane * 16) & pmask, g_kv, pg);
            }
            __syncwarp();
            looks += look;
          } else {
            const uint8_t* from = (is_v ? p.c.v : p.c.k) + g_kv * (is_v ? p.c.vs[2] : p.c.ks[2]);
            const int64_t sp = is_v ? p.c.vs[0] : p.c.ks[0], st = is_v ? p.c.vs[1] : p.c.ks[1];
            const int64_t group = static_cast<int64_t>(pg) * sp + ((j0 + (lane & 7) * 16) & pmask) * st;
            const uint8_t* mine = from + (r0 & 15) * st + chunk * 16;
            constexpr int PER = 16 / RPP;  // copies of a group of 16 keys
            uint32_t dst = smem_u32(to) + tile_off(r0, chunk);
#pragma unroll 1
            for (int g = 0; g < 8; ++g) {
              const uint8_t* src = mine + __shfl_sync(0xffffffffu, group, g);
              const bool paged = __shfl_sync(0xffffffffu, pg, g) >= 0;
#pragma unroll
              for (int i = 0; i < PER; ++i) {
                const int j = j0 + g * 16 + i * RPP + r0;
                const bool in = paged && (j < sink_hi || (j >= lo && j < hi));
                cp_async16(dst, in ? src : p.c.k, in ? cb : 0u);
                src += RPP * st;
                dst += RPP * 128;
              }
            }
            cp_async_wait_all();
            if (look && mend_pieces_apart<false>(smem_u32(to) + tile_off(r0, chunk), RPP * 128, NP, j0 + r0, RPP,
                                           part_seen(s, p.sinks)))
              s.odd = 1;
            announce(bar);
          }
          at.step();
        } else {
          // ---- the warp's 16 rows become bf16
          const int tile = it >> 1, place = it % kRaw;
          if (!is_v && !(ok = wait_all(cScale + tile % kScales, (tile / kScales) & 1))) break;
          if (!(ok = wait_all(cRaw + place, (it / kRaw) & 1) && slot_free(it))) break;
          const uint32_t src = raw + place * (128 * D);
          const uint8_t* exps = smem + L::kOffScale + tile % kScales * 256 + is_v * 128 + r0;
          const bool here = !((reinterpret_cast<const int*>(smem + L::kOffAbsent)[place] >> (warp - 12)) & 1);
          if (look && here && mend_pieces_apart<true, NB>(src, 512, NP, j0 + r0, RPP, part_seen(s, p.sinks))) s.odd = 1;
          // (loads of four pieces together: one after the other, each waited for the last one's store)
#pragma unroll
          for (int i4 = 0; i4 < NP; i4 += NB) {
            uint4 x4[NB];
#pragma unroll
            for (int i = 0; i < NB; ++i) {
              x4[i] = make_uint4(0u, 0u, 0u, 0u);
              if (here)
                asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
                             : "=r"(x4[i].x), "=r"(x4[i].y), "=r"(x4[i].z), "=r"(x4[i].w)
                             : "r"(src + (i4 + i) * 512)
                             : "memory");
            }
#pragma unroll
            for (int i = i4; i < i4 + NB; ++i) {
              // (the lanes of one row that lie 128 bytes apart in the tile's row store their halves in
              // opposite order: else every store would meet a second one in its banks)
              const bool turn = chunk >= 4;
              uint4 x = x4[i - i4];
              if (turn) x = make_uint4(x.z, x.w, x.x, x.y);
              const float sc = exp_scale(exps[i * RPP]);
              const uint64_t sc2 = f2(sc, sc);
              const uint32_t w[4] = {x.x, x.y, x.z, x.w};
              uint32_t o[8];
#pragma unroll
              for (int h = 0; h < 4; ++h) e4m3x4_to_f16x4(w[h], o[2 * h], o[2 * h + 1]);
#pragma unroll
              for (int h = 0; h < 8; ++h) {
                float a, c;
                asm("{\n\t.reg .b16 x, y;\n\tmov.b32 {x, y}, %2;\n\tcvt.f32.f16 %0, x;\n\tcvt.f32.f16 %1, y;\n\t}"
                    : "=f"(a), "=f"(c)
                    : "r"(o[h]));
                f2split(mul2(f2(a, c), sc2), a, c);
                o[h] = pack_bf16x2(a, c);
              }
#pragma unroll
              for (int h = 0; h < 2; ++h)
                *reinterpret_cast<uint4*>(sR + at.slot * L::kTile + tile_off(i * RPP + r0, chunk * 2 + (h ^ turn))) =
                    make_uint4(o[4 * h], o[4 * h + 1], o[4 * h + 2], o[4 * h + 3]);
            }
          }
          announce(cFull + at.slot);
          if (lane == 0) {
            mbar_arrive(&bars[cRawFree + place]);
            if (is_v) mbar_arrive(&bars[cScaleFree + tile % kScales]);
          }
          at.step();
        }
        ++it;
        // ---- the part's Q, behind its first loads
        if (i2 == (FP8 ? 0 : 1)) {
          if (idx > 0 && !(ok = wait_all(cQEmpty, (idx - 1) & 1))) break;
          constexpr int QCPR = D / 8;
          const int qc = lt % QCPR, row0 = s.row0, q0 = s.q0, h0 = s.g * p.G, rows = s.nq * p.G - row0;
          const uint32_t qb = qc * 8 < p.c.d ? 16u : 0u;
          // row row0 + r is (token, head) number first + r from the token of row0: a small number, so
          // the quotient by the group's size comes from one fp32 product (exact: checked for every
          // group size below 4096)
          const int tok0 = row0 / p.G, first = row0 - tok0 * p.G;
          const float by_g = 1.f / static_cast<float>(p.G);
#pragma unroll 4
          for (int r = lt / QCPR; r < 256; r += LT / QCPR) {
            const int x = first + r, i = p.G < 4096 ? static_cast<int>((static_cast<float>(x) + 0.5f) * by_g) : x / p.G;
            const uint32_t nb = r < rows ? qb : 0u;
            cp_async16(smem_u32(sQ) + (r >> 7) * L::kTile + tile_off(r & 127, qc),
                       nb ? p.q + (q0 + tok0 + i) * p.q_t + (h0 + x - i * p.G) * p.q_h + qc * 8 : p.q, nb);
          }
          cp_async_wait_all();
          announce(cQFull);
        }
      }
      if (!ok || n == 0) break;
      part_done(idx);
    }
    cp_async_wait_all();
    if (!FP8 && ok && lt == 0) {
      look_at[looks % kLooks] = Look{-1, 0, 0};
      mbar_arrive(&bars[cLook + looks % kLooks]);
    }
    // (after a time-out: the TMA boxes in flight land before the CTA ends)
    if (!FP8 && *abort_flag && warp == 12) {
      for (int i = max(looks - kLooks, 0); i < looks; ++i)
        mbar_wait(&bars[cLook + i % kLooks], (i / kLooks) & 1, p.err, kDevErrTimeout, nullptr);
      for (int i = 0; i < L::kRing && i < it; ++i) {
        at.phase ^= at.slot == 0 ? 1u : 0u;
        at.slot = at.slot == 0 ? L::kRing - 1 : at.slot - 1;
        mbar_wait(&bars[cFull + at.slot], at.phase, p.err, kDevErrTimeout, nullptr);
      }
    }
  } else if (warp < 4) {
    regs_decrease<Roles::kRegsMma>();
    if (warp == 0) {
      // ---------------------------------------------------------------- products
      // The whole warp runs the loop and one elected lane issues: the descriptors then stay in
      // uniform registers (with one lane running it all, a product took twice as long to issue).
      const bool one = elect_one();
      const uint64_t qd0 = sdesc_sw128(smem_u32(sQ), 16, 1024);
      const uint64_t kd0 = sdesc_sw128(smem_u32(sR), 16, 1024);      // K-major view of ring slot 0
      const uint64_t vd0 = sdesc_sw128(smem_u32(sR), 16384, 1024);   // MN-major view
      constexpr uint64_t step = static_cast<uint64_t>(L::kTile >> 4);
      Ring at;             // the next item to arrive: K_0, V_0, K_1, V_1, ...
      uint32_t np = 0;  // parity of the P tiles consumed by each slot
      int nparts[2] = {0, 0};
      bool ok = true;
      auto arrived = [&]() {
        if (!wait(cFull + at.slot, at.phase)) return false;
        tc_fence_after();
        return true;
      };
      auto issue_s = [&](int w, int slot) {
        if (!one) return;
        const uint64_t kd = kd0 + slot * step, qd = qd0 + w * step;
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          const uint64_t off = static_cast<uint64_t>(((k >> 2) * 16384u + (k & 3) * 32u) >> 4);
          umma_ss(tbase + w * 128, qd + off, kd + off, IDESC_S, k > 0);
        }
        umma_commit(&bars[cSFull + w]);
      };
      auto pv = [&](int w, int slot, bool start) {
        // O_w holds the slot's previous part until its rows have read it
        if (start && nparts[w] > 1 && !wait(cOFree + w, nparts[w] & 1)) return false;
        const uint64_t vd = vd0 + slot * step;
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          if (!wait(cPReady + 2 * w + hf, (np >> w) & 1u)) return false;
          tc_fence_after();
          if (!one) continue;
#pragma unroll
          for (int k = hf * 4; k < hf * 4 + 4; ++k)
            umma_ts(tbase + 256 + w * 128, tbase + w * 128 + k * 8, vd + static_cast<uint64_t>((k * 2048) >> 4), IDESC_O,
                    (!start || k > 0) ? 1u : 0u);
        }
        np ^= 1u << w;
        return true;
      };
      for (int idx = 0; ok; ++idx) {
        if (!(ok = part_ready(idx))) break;
        const int n = parts[idx % kParts].n;
        const bool both = parts[idx % kParts].slots == 2;
        if (one) part_done(idx);
        if (n == 0) break;
        ++nparts[0];
        if (!(ok = wait(cQFull, idx & 1))) break;
        // (a loop for each number of slots: with one for both, a 2048-token chunk took 177 instead of 173 us)
        if (both) {
          ++nparts[1];
          for (int k = 0; ok && k <= n; ++k) {
            int vslot = 0, kslot = 0;
            if (k > 0) {
              if (!(ok = arrived())) break;
              vslot = at.slot;
              at.step();
            }
#pragma unroll
            for (int w = 0; w < 2; ++w) {
              if (k > 0) {
                if (!(ok = pv(w, vslot, k == 1))) break;
                if (w == 1 && one) umma_commit(&bars[cEmpty + vslot]);
                if (k == n && one) umma_commit(&bars[cOFinal + w]);
              }
              if (k < n) {
                if (w == 0) {
                  if (!(ok = arrived())) break;
                  kslot = at.slot;
                  at.step();
                }
                issue_s(w, kslot);
              }
            }
            if (ok && k < n && one) umma_commit(&bars[cEmpty + kslot]);
            if (ok && k == n - 1 && one) umma_commit(&bars[cQEmpty]);
          }
        } else {
#pragma unroll 1
          for (int k = 0; ok && k <= n; ++k) {
            if (k > 0) {
              if (!(ok = arrived() && pv(0, at.slot, k == 1))) break;
              if (one) umma_commit(&bars[cEmpty + at.slot]);
              if (k == n && one) umma_commit(&bars[cOFinal]);
              at.step();
            }
            if (k < n) {
              if (!(ok = arrived())) break;
              issue_s(0, at.slot);
              if (one) umma_commit(&bars[cEmpty + at.slot]);
              if (k == n - 1 && one) umma_commit(&bars[cQEmpty]);
              at.step();
            }
          }
        }
      }
      __syncwarp();
      if (one) umma_commit(&bars[cDrain]);
      mbar_wait(&bars[cDrain], 0, p.err, kDevErrTimeout, nullptr);
    } else if (FP8 && warp < 3) {
      // ------------------------------------------------- e4m3: codes (warp 1) and scale bytes (warp 2)
      const int pmask = (1 << p.c.page_shift) - 1, sub = warp == 1 ? (lane & 7) * 16 : lane * 4;
      uint8_t* const raw = smem + L::kOffRaw;
      int tile = 0, issued = 0;  // tiles so far in the run; items on their way
      bool ok = true;
      for (int idx = 0; ok; ++idx) {
        if (!(ok = part_ready_all(idx))) break;
        const Part& s = parts[idx % kParts];
        const int n = s.n, b = s.b, g = s.g, lo = s.lo, hi = s.hi, sink_hi = s.sink_hi;
        const PartTiles tiles(s);
        __syncwarp();
        if (lane == 0) part_done(idx);
        if (n == 0) break;
        // the page of this lane's keys of a tile, looked up one tile ahead; none where no row sees a key
        // of the group of 16
        auto look_up = [&](int k) {
          int entry = kNoKeys;
          if (k < n) {
            const int j = tiles.key0(k) + (sub & -16);
            if (j < sink_hi || (j < hi && j + 16 > lo)) entry = table_entry(p, b, j);
          }
          return entry;
        };
        int next = look_up(0);
#pragma unroll 1
        for (int k = 0; ok && k < n; ++k, ++tile) {
          const int j = tiles.key0(k) + sub, pg = checked_page(p, next);
          next = look_up(k + 1);
          if (warp == 1) {
            const unsigned here = __ballot_sync(0xffffffffu, lane < 8 && pg >= 0);
#pragma unroll 1
            for (int is_v = 0; is_v < 2; ++is_v) {
              const int it = 2 * tile + is_v, place = it % kRaw;
              if (it >= kRaw && !(ok = wait_all(cRawFree + place, (it / kRaw - 1) & 1))) break;
              uint8_t* to = raw + place * (128 * D);
              uint64_t* bar = &bars[cRaw + place];
              if (lane == 0) {
                reinterpret_cast<unsigned*>(smem + L::kOffAbsent)[place] = ~here;
                if (p.box > 0) mbar_arrive_expect_tx(bar, __popc(here) * 16 * D);
              }
              __syncwarp();
              if (p.box > 0) {
                if ((here >> lane) & 1u) tma_load_4d(to + lane * 16 * D, is_v ? &tmV : &tmK, bar, 0, j & pmask, g, pg);
              } else {
                constexpr int CPR = D / 16;
                const int64_t* st = is_v ? p.c.vs : p.c.ks;
                const uint8_t* from = (is_v ? p.c.v : p.c.k) + g * st[2];
#pragma unroll 1
                for (int i = lane; i < 128 * CPR; i += 32) {
                  const int grp = i / (16 * CPR), page = __shfl_sync(0xffffffffu, pg, grp);
                  const int slot = (__shfl_sync(0xffffffffu, j, grp) & pmask) + i / CPR % 16, c = i % CPR * 16;
                  if (page >= 0)
                    cp_async16(smem_u32(to) + i * 16, c < p.c.d ? from + page * st[0] + slot * st[1] + c : p.c.k,
                               c < p.c.d ? 16u : 0u);
                }
                cp_async_wait_all();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar);
              }
              ++issued;
            }
          } else {
            uint32_t e[2] = {0x7f7f7f7fu, 0x7f7f7f7fu};
            if (pg >= 0) {
              uint32_t x[2][4];
#pragma unroll
              for (int is_v = 0; is_v < 2; ++is_v) {
                const int64_t* st = is_v ? p.c.ves : p.c.kes;
                const uint8_t* from = (is_v ? p.c.ve : p.c.ke) + g * st[2] + pg * st[0] + (j & pmask) * st[1];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                  x[is_v][i] = 127;
                  if (j + i < sink_hi || (j + i >= lo && j + i < hi)) x[is_v][i] = from[i * st[1]];
                }
              }
#pragma unroll
              for (int is_v = 0; is_v < 2; ++is_v)
                e[is_v] = scale_byte(x[is_v][0]) | scale_byte(x[is_v][1]) << 8 | scale_byte(x[is_v][2]) << 16 |
                          scale_byte(x[is_v][3]) << 24;
            }
            const int place = tile % kScales;
            if (tile >= kScales && !(ok = wait_all(cScaleFree + place, (tile / kScales - 1) & 1))) break;
            uint32_t* to = reinterpret_cast<uint32_t*>(smem + L::kOffScale + place * 256) + lane;
            to[0] = e[0];
            to[32] = e[1];
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars[cScale + place]);
          }
        }
      }
      cp_async_wait_all();
      // (the boxes in flight land before the CTA ends, after a time-out too)
      if (warp == 1) {
        for (int i = max(issued - kRaw, 0); i < issued; ++i)
          mbar_wait(&bars[cRaw + i % kRaw], (i / kRaw) & 1, p.err, kDevErrTimeout, nullptr);
      }
    } else if (!FP8 && warp < 3) {
      // ---------------------------------------------------------------- looking
      constexpr int CPR = D / 8, RPP = 64 / CPR;
      const int chunk = (tid - 32) % CPR, r0 = (tid - 32) / CPR;
      // (rows eight apart have a column of pieces at equal distances)
      for (int i = 0;; ++i) {
        if (!__all_sync(0xffffffffu, idle_wait(cLook + i % kLooks, (i / kLooks) & 1))) break;
        const Look k = look_at[i % kLooks];
        if (k.slot < 0) break;
        Part& s = parts[k.part % kParts];
        const SeenKeys seen = part_seen(s, p.sinks);
        bool found = false;
#pragma unroll 1
        for (int r = r0; r < 8; r += RPP)
          found |= mend_pieces<false>(smem_u32(sR) + k.slot * L::kTile + tile_off(r, chunk), 1024, 16, k.j0 + r, 8, seen);
        if (found) s.odd = 1;
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&bars[cFull + k.slot]);
          mbar_arrive(&bars[cFull + k.slot]);
        }
      }
    } else if (warp == 3 && lane == 0) {
      // ---------------------------------------------------------------- walk
      for (int left = c.left, idx = 0;; ++idx) {
        if (idx >= kParts && !idle_wait(cPartFree + idx % kParts, (idx / kParts - 1) & 1)) break;
        Part& s = parts[idx % kParts];
        s.n = max(min(c.r.tiles - c.t, left), 0);
        if (left > 0) {
          s.whole = s.n == c.r.tiles;
          s.slot = idx == 0 ? 0 : 1;
          s.row0 = c.rt * ROWS;
          s.slots = c.s.nq * p.G - s.row0 > 128 ? 2 : 1;
          s.t0 = c.t;
          s.sink_tiles = c.r.sink_tiles;
          s.main0 = c.r.main0;
          s.lo = c.r.lo;
          s.hi = c.r.hi;
          s.sink_hi = c.r.sink_hi;
          s.b = c.b;
          s.g = c.g;
          s.q0 = c.s.q0;
          s.nq = c.s.nq;
          s.pos0 = c.s.pos0;
          s.klen = c.s.klen;
          const int i0 = s.row0 / p.G, i1 = min((s.row0 + ROWS - 1) / p.G, s.nq - 1);
          s.all_hi = row_keys(p, c.s, c.s.pos0 + i0).hi;
          s.all_lo = row_keys(p, c.s, c.s.pos0 + i1).lo;
          s.odd = 0;
        }
        mbar_arrive(&bars[cPart + idx % kParts]);
        if (left <= 0) break;
        if (c.t == 0 && !s.whole)
          p.desc[blockIdx.x] =
              make_int4(c.b, c.g, c.rt, s.slot | (1 + (c.r.tiles - s.n + quota - 1) / quota) << 1);
        const int n = s.n;
        left -= n + (c.t + n == c.r.tiles ? kItemCost : 0);
        c.t += n - 1;
        if (left > 0) c.next(p);
      }
    }
  } else {
    // -------------------------------------------------------------------- softmax
    regs_increase<Roles::kRegsSoft>();
    const int w = (warp >> 2) - 1, quad = warp & 3, row = w * 128 + quad * 32 + lane;
    const uint32_t tl = tbase + (static_cast<uint32_t>(quad * 32) << 16);
    const uint32_t scol = w * 128, ocol = 256 + w * 128;
    const float cexp = p.scale_log2;
    const uint64_t c2 = f2(cexp, cexp);
    uint32_t parity = 0;  // of this slot's S tiles (bit 0) and parts (bit 1) so far
    bool ok = true;
    for (int idx = 0; ok; ++idx) {
      if (!(ok = part_ready_all(idx))) break;
      const Part& s = parts[idx % kParts];
      const int n = s.n;
      if (n == 0) break;
      if (w < s.slots) {
        // (a row past the item's last one is treated like the last: nothing is stored for it)
        const int R = s.row0 + row, last = s.nq * p.G - 1;
        const int pos = s.pos0 + min(R, last) / p.G;
        const int rhi = p.causal ? pos + 1 : s.klen, rlo = p.window > 0 ? pos - p.window + 1 : 0;
        float m = kNInf, l = 0.f;
        for (int k = 0; k < n; ++k, parity ^= 1u) {
          const int j0 = PartTiles(s).key0(k);  // (not kept: there is no register to spare here)
          const int hi = rhi - j0, lo = rlo - j0, sk = p.sinks - j0;
          const bool masked = !__all_sync(0xffffffffu, hi >= 128 && (lo <= 0 || sk >= 128));
          if (!(ok = wait_all(cSFull + w, parity & 1u))) break;
          tc_fence_after();
          auto mask32 = [&](int a, uint32_t (&x)[32]) {
            auto below = [](int n) { return n <= 0 ? 0u : n >= 32 ? 0xffffffffu : (1u << n) - 1u; };
            const uint32_t see = below(hi - a * 32) & (~below(lo - a * 32) | below(sk - a * 32));
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if (!((see >> e) & 1u)) x[e] = 0xff800000u;
          };
          auto max32 = [](const uint32_t (&x)[32]) {
            float t = __uint_as_float(x[0]);
            asm("max.f32 %0, %0, %1;" : "+f"(t) : "f"(__uint_as_float(x[1])));
#pragma unroll
            for (int e = 2; e < 32; e += 2)
              asm("max.f32 %0, %0, %1, %2;" : "+f"(t) : "f"(__uint_as_float(x[e])), "f"(__uint_as_float(x[e + 1])));
            return t;
          };
          // bf16: the row's 128 scores stay in registers.  e4m3: they are read from TMEM twice, 64 at a
          // time, which leaves registers for more loading warps.
          uint32_t x[FP8 ? 2 : 4][32];
          float mx = kNInf;
          auto load64 = [&](int a) {
            tmem_ld32(tl + scol + a * 32, x[0]);
            tmem_ld32(tl + scol + a * 32 + 32, x[1]);
            tmem_ld_wait(x[0]);
            tmem_ld_tie(x[1]);
            if (masked) {
              mask32(a, x[0]);
              mask32(a + 1, x[1]);
            }
          };
          if (FP8) {
#pragma unroll 1
            for (int a = 0; a < 4; a += 2) {
              load64(a);
              mx = fmaxf(mx, fmaxf(max32(x[0]), max32(x[1])));
            }
          } else {
#pragma unroll
            for (int a = 0; a < 4; ++a) tmem_ld32(tl + scol + a * 32, x[FP8 ? 0 : a]);
            tmem_ld_wait(x[0]);
#pragma unroll
            for (int a = 1; a < 4; ++a) tmem_ld_tie(x[FP8 ? 0 : a]);
            if (masked) {
#pragma unroll
              for (int a = 0; a < 4; ++a) mask32(a, x[FP8 ? 0 : a]);
            }
            float mx4[4];
#pragma unroll
            for (int a = 0; a < 4; ++a) mx4[a] = max32(x[FP8 ? 0 : a]);
            mx = fmaxf(fmaxf(mx4[0], mx4[1]), fmaxf(mx4[2], mx4[3]));
          }
          const float mn = fmaxf(m, mx);
          float alpha = 1.f;
          if ((mn - m) * cexp > kRaise) {  // (also from -inf)
            alpha = m == kNInf ? 0.f : paged_ex2((m - mn) * cexp);
            l *= alpha;
            m = mn;
          }
          if (k > 0 && __any_sync(0xffffffffu, alpha != 1.f)) {
            // S_w of this tile was issued after the PV_w of the last one, and the next PV_w waits
            // for the arrivals below: O_w is at rest
#pragma unroll
            for (int a = 0; a < D / 16; ++a) {
              uint32_t o16[16];
              tmem_ld16(tl + ocol + a * 16, o16);
              tmem_ld_wait(o16);
#pragma unroll
              for (int e = 0; e < 16; ++e) o16[e] = __float_as_uint(__uint_as_float(o16[e]) * alpha);
              tmem_st16(tl + ocol + a * 16, o16);
            }
          }
          const float nm = m == kNInf ? 0.f : -(m * cexp);
          const uint64_t nm2 = f2(nm, nm);
          uint64_t sum[2] = {0ull, 0ull};
          auto weights32 = [&](int a, const uint32_t (&x)[32]) {
            uint32_t pk[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              float e0, e1;
              f2split(fma2(f2(__uint_as_float(x[2 * e]), __uint_as_float(x[2 * e + 1])), c2, nm2), e0, e1);
              e0 = paged_ex2(e0);
              e1 = paged_ex2(e1);
              sum[e & 1] = add2(sum[e & 1], f2(e0, e1));
              pk[e] = pack_bf16x2(e0, e1);
            }
            tmem_st16(tl + scol + a * 16, pk);
            if (a & 1) {  // keys 0..63, then 64..127
              tmem_st_wait();
              tc_fence_before();
              mbar_arrive(&bars[cPReady + 2 * w + (a >> 1)]);
            }
          };
          if (FP8) {
#pragma unroll 1
            for (int a = 0; a < 4; a += 2) {
              load64(a);
              weights32(a, x[0]);
              weights32(a + 1, x[1]);
            }
          } else {
#pragma unroll
            for (int a = 0; a < 4; ++a) weights32(a, x[FP8 ? 0 : a]);
          }
          float s0, s1;
          f2split(add2(sum[0], sum[1]), s0, s1);
          l += s0 + s1;
        }
        if (!ok) break;
        // ---- the part's end
        if (!(ok = wait_all(cOFinal + w, parity >> 1))) break;
        parity ^= 2u;
        tc_fence_after();
        const bool real = R <= last, whole = s.whole, odd = *const_cast<volatile int*>(&s.odd) != 0;
        const int tok = real ? R / p.G : 0;
        const float inv = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);
        const int64_t pb = (static_cast<int64_t>(blockIdx.x) * 2 + s.slot) * ROWS;
        const int h = s.g * p.G + R - tok * p.G;
        const int64_t t = s.q0 + tok;
#pragma unroll
        for (int a = 0; a < D / 32; ++a) {
          uint32_t o[32];
          tmem_ld32(tl + ocol + a * 32, o);
          tmem_ld_wait(o);
          if (whole) {
            uint16_t* dst = p.out + (t * p.Hq + h) * p.c.d + a * 32;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              uint32_t pk[4];
#pragma unroll
              for (int i = 0; i < 4; ++i)
                pk[i] = pack_bf16x2(__uint_as_float(o[e * 8 + 2 * i]) * inv, __uint_as_float(o[e * 8 + 2 * i + 1]) * inv);
              if (real && a * 32 + e * 8 < p.c.d)
                *reinterpret_cast<uint4*>(dst + e * 8) = make_uint4(pk[0], pk[1], pk[2], pk[3]);
            }
          } else {
            // [column / 4][row]: a warp's stores are contiguous
#pragma unroll
            for (int e = 0; e < 8; ++e)
              reinterpret_cast<uint4*>(p.part_o)[pb * (D / 4) + (a * 8 + e) * ROWS + row] =
                  make_uint4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
          }
        }
        tc_fence_before();
        mbar_arrive(&bars[cOFree + w]);
        if (odd && real) {
          const int mid = min(s.all_lo, s.hi);
          const OddKeys k{s.b,  s.g,  s.lo, mid, max(max(s.all_hi, s.lo), mid), s.hi, s.sink_tiles, s.main0,
                          s.t0, s.t0 + n - 1};
          add_odd_values<FP8, kKeyTile>(p, k, rlo, rhi, 0, p.c.d, whole ? p.out + (t * p.Hq + h) * p.c.d : nullptr,
                                        p.part_o + (pb * (D / 4) + row) * 4, ROWS * 4);
        }
        if (whole) {
          if (real) p.lse[static_cast<int64_t>(h) * p.T + t] = l == 0.f ? kNInf : (m * cexp + log2f(l)) * kPLn2;
        } else {
          p.part_ml[pb + row] = make_float2(m == kNInf ? m : m * cexp, l);
        }
      }
      part_done(idx);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tbase, 512);
  }
}

template <int D, bool FP8>
cudaError_t launch_chunk(PagedParams p, cudaStream_t stream) {
  using L = ChunkSmem<D, FP8>;
  auto kern = paged_chunk_kernel<D, FP8>;
  static std::atomic<uint64_t> ready{0};
  cudaError_t e = set_up_once(ready, kern, L::kTotal, ChunkRoles<FP8>::kLaunchRegs);  // (the setmaxnreg split must fit)
  if (e != cudaSuccess) return e;
  CUtensorMap tk{}, tv{};
  const int page = 1 << p.c.page_shift, rows = FP8 ? 16 : page < 128 ? page : 128, cols = FP8 ? D : 64;
  // (a cache that broadcasts an axis with stride 0 goes by cp.async)
  p.box = paged_map(&tk, FP8, p.c.k, p.c.d, page, p.c.Hkv, p.c.num_pages, p.c.ks, cols, rows) &&
                  paged_map(&tv, FP8, p.c.v, p.c.d, page, p.c.Hkv, p.c.num_pages, p.c.vs, cols, rows)
              ? rows
              : 0;
  kern<<<kPagedCtas, ChunkRoles<FP8>::kThreads, L::kTotal, stream>>>(tk, tv, p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_paged_chunk(bool fp8, const PagedParams& p, cudaStream_t stream) {
  if (p.c.d <= 64) return fp8 ? launch_chunk<64, true>(p, stream) : launch_chunk<64, false>(p, stream);
  return fp8 ? launch_chunk<128, true>(p, stream) : launch_chunk<128, false>(p, stream);
}

}  // namespace fdma
