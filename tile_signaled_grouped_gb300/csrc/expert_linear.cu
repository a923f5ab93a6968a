// The experts' matrix products on tcgen05: rows sorted by expert, each expert with its own weights.
//
//   forward   y[r]  = W[e] x[r]             rows r of expert e: offsets[e] .. offsets[e + 1] - 1
//   backward  dx[r] = W[e]^T dy[r] + add[r]
//             dW[e] = sum over e's rows of dy[r] x[r]^T
//
// How many rows an expert has is known on the device only, and is uneven. So the rows are the columns
// of the products y^T = W x^T and dx^T = W^T dy^T, whose number a tcgen05.mma takes in steps of 32, and the
// 256 features of a CTA pair's tile are its rows: an expert with 40 rows costs 64 columns where it would
// cost a whole tile of 128 or 256 rows. In dW the rows are summed over, 64 at a time, and those past an expert's
// last are zeroed in shared memory.
#include <algorithm>
#include <atomic>
#include <type_traits>

#include "mma_common.cuh"

namespace moe {
namespace {

constexpr int kMaxExperts = 1024;
constexpr int kMaxStages = 8;
constexpr int kEpiWarps = 8;
constexpr int kThreads = 32 * (2 + kEpiWarps);
constexpr int kFeatures = 256;                  // of a pair's tile
constexpr int kRows = 256;                      // of a pair's tile at most
constexpr int kRowStep = 32;                    // columns of a product come in this step
constexpr int kGroup = 8;                       // tiles of rows that walk the features together
constexpr int kABytes = 128 * 128;              // a CTA's features of a block of 64 k
constexpr int kBlockBytes = kABytes + 128 * 128;  // and half of the pair's rows
constexpr int kPatchBytes = 32 * 64;            // of an epilogue warp: 32 rows of 64 bytes
constexpr int kWeightEpiWarps = 16;             // dW: its epilogues have most to write
constexpr int kWeightThreads = 32 * (3 + kWeightEpiWarps);

struct PairSmem {
  uint64_t full[kMaxStages], empty[kMaxStages];
  uint64_t tfull[2], tempty[2];
  uint64_t drain;
  uint64_t last[kMaxStages];  // dW: this CTA's copies of a block with rows past the expert's last
  uint32_t tmem;
  int abort;
  int scratch[33];
};

__device__ __forceinline__ void tma_load_3d_pair(void* dst, const CUtensorMap* map, uint32_t cl_bar, int x,
                                                 int y, int z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%3, %4, %5}], [%2];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(cl_bar), "r"(x), "r"(y), "r"(z)
      : "memory");
}

// Piece `k` (16 bytes) of row r of a patch: eight lanes that take one piece of eight rows each, or four of
// two, meet no bank twice.
__device__ __forceinline__ int patch_at(int r, int k) { return r * 64 + ((k ^ (r >> 1)) & 3) * 16; }

// 16 lanes x 32 columns of TMEM as 8 x 8 pieces: of the columns 8 i .. a thread has, in v[4 i], v[4 i + 1], the
// columns 2 (lane & 3) and the next of lane / 4, in the other two those of lane / 4 + 8.
__device__ __forceinline__ void tmem_ld_pieces(uint32_t taddr, uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]),
        "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
      : "r"(taddr));
}
// Four 8 x 8 pieces of 16 bits, each thread with two neighbours of a row as above, to or from shared memory
// turned round: lane l's address is that of column l & 7 of piece l >> 3.
__device__ __forceinline__ void store_turned(uint32_t addr, const uint32_t (&w)[4]) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared::cta.b16 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(w[0]),
               "r"(w[1]), "r"(w[2]), "r"(w[3])
               : "memory");
}
__device__ __forceinline__ void load_turned(uint32_t addr, uint32_t (&w)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared::cta.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
               : "r"(addr)
               : "memory");
}

// An epilogue warp has read its part of an accumulator: its loads are complete (tcgen05.wait::ld) and nothing
// else of it is the products' business, so the arrival orders no memory. (A release would wait for the warp's
// stores to the outputs before it: 656 us where this takes 513, dW of 128 experts of 64 rows, 2048 x 4096.)
__device__ __forceinline__ void arrive_read(uint32_t cl_addr) {
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(cl_addr) : "memory");
}

__device__ __forceinline__ void tma_store_3d(const CUtensorMap* map, const void* src, int x, int y, int z) {
  asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.bulk_group [%0, {%2, %3, %4}], [%1];" ::"l"(
                   reinterpret_cast<uint64_t>(map)),
               "r"(smem_u32(src)), "r"(x), "r"(y), "r"(z)
               : "memory");
}

__device__ __forceinline__ void tma_add_3d(const CUtensorMap* map, const void* src, int x, int y, int z) {
  asm volatile("cp.reduce.async.bulk.tensor.3d.global.shared::cta.add.bulk_group [%0, {%2, %3, %4}], [%1];" ::"l"(
                   reinterpret_cast<uint64_t>(map)),
               "r"(smem_u32(src)), "r"(x), "r"(y), "r"(z)
               : "memory");
}

// The rows of expert e, whatever the offsets hold inside 0 .. n; as e = E those behind the last expert's, as
// E + 1 those before the first's.
__device__ __forceinline__ void rows_of(const int32_t* offsets, int e, int E, int n, int* start, int* count) {
  const int lo = e <= E ? min(max(__ldg(offsets + e), 0), n) : 0;
  const int hi = e < E ? min(max(__ldg(offsets + e + 1), lo), n) : e == E ? n : min(max(__ldg(offsets), 0), n);
  *start = lo;
  *count = hi - lo;
}

// The barriers and the tensor memory of a pair; both CTAs have them when it returns.
// `full`: arrivals that fill a stage; `epi`: epilogue warps of a CTA.
__device__ __forceinline__ void pair_setup(PairSmem& sm, int stages, int warp, int full, int epi) {
  if (threadIdx.x == 0) {
    for (int i = 0; i < stages; ++i) {
      mbar_init(&sm.full[i], full);  // rank 0: its arrive.expect_tx (bytes of both CTAs) is one
      mbar_init(&sm.last[i], 1);
      mbar_init(&sm.empty[i], 1);  // the leader's commit (multicast)
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sm.tfull[i], 1);              // the leader's commit (multicast)
      mbar_init(&sm.tempty[i], 2 * epi);       // rank 0: both CTAs' epilogue warps
    }
    mbar_init(&sm.drain, 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    sm.abort = 0;
  }
  if (warp == 1) tmem_alloc_pair(&sm.tmem, 512);
  tc_fence_before();
  __syncthreads();
  __syncwarp();
  cluster_sync_all();
  tc_fence_after();
}
// Both CTAs meet: the leader's products (which read both CTAs' shared memory and write both
// CTAs' TMEM) are done, every copy has landed and every accumulator is read.
__device__ __forceinline__ void pair_teardown(uint32_t tmem, int warp) {
  tc_fence_before();
  __syncthreads();
  __syncwarp();
  cluster_sync_all();
  tc_fence_after();
  if (warp == 1) tmem_dealloc_pair(tmem, 512);
}
// The loads' warp, at its end: every copy this CTA issued has landed once the products that read its stage
// are done (with a limit).
__device__ __forceinline__ void wait_copies(PairSmem& sm, int issued, int stages, uint32_t* status) {
  volatile int never = 0;
  const unsigned long long t0 = globaltimer();
  for (int i = max(0, issued - stages); i < issued; ++i) {
    const long long left = kWaitNs - (long long)(globaltimer() - t0);
    pwait(&sm.empty[i % stages], (i / stages) & 1, &never, left > 0 ? left : 0, status, 0x42000000u);
  }
}
// The products' warp, at its end: every product issued is done.
__device__ __forceinline__ void wait_products(PairSmem& sm, uint32_t* status) {
  if (elect_one()) tc_commit_pair(&sm.drain, 0x1);
  __syncwarp();
  volatile int never = 0;
  pwait(&sm.drain, 0, &never, kWaitNs, status, 0x43000000u);
}

// ------------------------------------------------------------------- y and dx
struct RowsArgs {
  CUtensorMap tw, tx[4];  // weights (3-D: experts outermost); 16, 32, 64 and 128 rows
  const int32_t* offsets;
  void* y;             // [n][ld_y]
  const void* add;     // [n][ld_add] or null
  long long ld_y, ld_add;
  uint32_t* status;
  int n, E, J, nk;     // J: features of y; nk: 64-element blocks of the sum
  int tiles_j, stages; // tiles_j: tiles of features times splits
  int most;            // tiles of rows at most
  int split_bits;      // 2^split_bits pairs share a tile, each with a range of the sum
  float* part;         // [splits][n][J], their sums, or null
  bool w_mn;           // W^T, whose features are innermost
};
constexpr int kBlocks = 2;  // of 64 k in a stage

// The table of the experts' rows in shared memory, entries E and E + 1 for the rows behind the last
// expert's and before the first's (zeros): first row, number, and the tiles of rows before it. An
// expert's rows are shared out evenly over its tiles.
struct Table {
  int *start, *count, *first;
  int tiles;  // of rows, all of them
};
__host__ __device__ constexpr size_t table_bytes(int E) { return (size_t)(3 * (E + 2) + 3) / 4 * 16; }
__device__ __forceinline__ Table make_table(const RowsArgs& a, int* at, int* scratch) {
  Table t{at, at + a.E + 2, at + 2 * (a.E + 2), 0};
  constexpr int kEach = (kMaxExperts + 1 + kThreads) / kThreads;  // neighbouring entries a thread
  int tiles[kEach], sum = 0;
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    const int e = threadIdx.x * kEach + i;
    tiles[i] = 0;
    if (e <= a.E + 1) {
      int start, count;
      rows_of(a.offsets, e, a.E, a.n, &start, &count);
      t.start[e] = start;
      t.count[e] = count;
      tiles[i] = (count + kRows - 1) / kRows;
    }
    sum += tiles[i];
  }
  int at_tile = block_excl_scan(sum, scratch, &t.tiles);
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    const int e = threadIdx.x * kEach + i;
    if (e <= a.E + 1) t.first[e] = at_tile;
    at_tile += tiles[i];
  }
  t.tiles = min(t.tiles, a.most);
  __syncthreads();
  return t;
}

// x / d for d = 1 .. 8 and x below 2^29: the product with 2^32 / d rounded up is off by less than x d.
__constant__ uint32_t kInverse[9] = {0,          0,          0x80000000u, 0x55555556u, 0x40000000u,
                                     0x33333334u, 0x2AAAAAABu, 0x24924925u, 0x20000000u};
__device__ __forceinline__ int small_quotient(int x, int d) {
  return d <= 1 ? x : (int)__umulhi((uint32_t)x, kInverse[d]);
}

// The tiles of a pair: p, p + pairs, ... of the order expert, feature tile, tile of rows, so that
// tiles that share their weights are neighbours. Every role of both CTAs walks the same, as whole warps:
// with a search by one thread and five divisions a tile took each of them 1400 cycles, more than the
// products of a short sum.
struct RowWalk {
  const RowsArgs& a;
  const Table& t;
  int tile, part;        // tile of rows among all experts', and the rest: the position is tile * tiles_j + part
  int step_tile, step_part;
  int e, j0, row0, rows, cols;  // the tile: expert, first feature, first row, rows, rows rounded up
  int split, k0, k1;            // which part of the sum, its blocks

  __device__ __forceinline__ RowWalk(const RowsArgs& args, const Table& table, int pair, int n)
      : a(args), t(table), e(0), j0(0), row0(0), rows(0), cols(0), split(0), k0(0), k1(0) {
    step_tile = n / a.tiles_j;
    step_part = n - step_tile * a.tiles_j;
    tile = pair / a.tiles_j - step_tile;
    part = pair - pair / a.tiles_j * a.tiles_j - step_part;
  }
  __device__ __forceinline__ bool next() {
    const int lane = threadIdx.x & 31;
    constexpr int kSpan = (kMaxExperts + 1 + 32) / 32;  // entries of a lane in the first of two steps: 33
    while (true) {
      tile += step_tile;
      part += step_part;
      if (part >= a.tiles_j) {
        part -= a.tiles_j;
        ++tile;
      }
      if (tile >= t.tiles) return false;
      // The last expert whose first tile is not past it.
      const int last = a.E + 1;
      const bool at = lane * kSpan <= last && t.first[min(lane * kSpan, last)] <= tile;
      const int base = (31 - __clz((int)(__ballot_sync(kAll, at) | 1u))) * kSpan, mine = base + 1 + lane;
      const bool in = mine <= last && t.first[min(mine, last)] <= tile;
      e = min(base + __popc(__ballot_sync(kAll, in)), last);
      // Groups of kGroup tiles of rows, inside a group feature by feature: the tiles in flight share their
      // operands in L2 (all tiles of rows of a feature tile first took 185 us where this takes 149 for 16384
      // rows of one expert, 2048 x 4096). Up to kGroup tiles share an expert's rows evenly, which is as far as
      // the quotient goes; of more the last alone is shorter.
      const int count = t.count[e], tiles = (count + kRows - 1) / kRows;
      int local = (tile - t.first[e]) * a.tiles_j + part, from = 0, in_group = tiles, per = kRows;
      if (tiles <= kGroup) {
        per = (small_quotient(count + tiles - 1, tiles) + kRowStep - 1) / kRowStep * kRowStep;
      } else {
        const int g = local / (kGroup * a.tiles_j);
        local -= g * kGroup * a.tiles_j;
        from = g * kGroup;
        in_group = min(kGroup, tiles - from);
      }
      const int tj = small_quotient(local, in_group), ti = from + local - tj * in_group;
      j0 = (tj >> a.split_bits) * kFeatures;
      split = tj & ((1 << a.split_bits) - 1);
      k0 = (int)((long long)a.nk * split >> a.split_bits);
      k1 = (int)((long long)a.nk * (split + 1) >> a.split_bits);
      row0 = t.start[e] + ti * per;
      rows = min(per, count - ti * per);
      cols = (rows + kRowStep - 1) / kRowStep * kRowStep;
      // (Offsets that do not ascend may make more tiles than an int counts: no rows then.)
      if (in_group > 0 && ti >= 0 && rows > 0) return true;
    }
  }
  __device__ __forceinline__ int steps() const { return e < a.E ? k1 - k0 : 0; }
};

// y = W x or dx = W^T dy + add. Bound by the weights' bytes for few rows of an expert (8 rows of 8 experts,
// 2048 x 7168: 42 us, 5.5 TB/s), by the products for many (8192 rows of 8, 8192 x 2048: 158 us, 1.74 PFLOP/s),
// and between the two by what crosses between the dies (32768 uneven rows of 128, 2048 x 4096: 465 to 505 us,
// 5.0 to 5.2 TB/s cross).
template <typename T>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    expert_rows_product_kernel(const __grid_constant__ RowsArgs a) {
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  uint8_t* base = smem_raw + (((raw + 1023u) & ~1023u) - raw);
  uint8_t* patches = base + (size_t)a.stages * kBlocks * kBlockBytes;
  int* table_at = reinterpret_cast<int*>(patches + kEpiWarps * kPatchBytes);
  PairSmem& sm = *reinterpret_cast<PairSmem*>(patches + kEpiWarps * kPatchBytes + table_bytes(a.E));
  constexpr bool kBf16 = std::is_same<T, __nv_bfloat16>::value;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t crank = cluster_ctarank();
  const bool lead = crank == 0;
  pair_setup(sm, a.stages, warp, 1, kEpiWarps);
  const uint32_t tmem = sm.tmem;
  wait_prior_grid();
  const Table table = make_table(a, table_at, sm.scratch);
  RowWalk walk(a, table, blockIdx.x >> 1, gridDim.x >> 1);

  if (warp == 0) {
    int n = 0, st = 0;
    uint32_t phase = 1;
    bool ok = true;
    while (ok && walk.next()) {
      const int j = walk.j0 + (int)crank * 128, half = walk.cols / 2;
      const int row = walk.row0 + (int)crank * half, steps = walk.steps();
      const uint32_t bytes = 2 * (kABytes + half * 128);
      for (int kb = 0; kb < steps; kb += kBlocks, ++n) {
        if (!warp_pwait(&sm.empty[st], phase, &sm.abort, a.status, 0x41000000u)) {
          ok = false;
          break;
        }
        if (elect_one()) {
          uint8_t* as = base + (size_t)st * (kBlocks * kBlockBytes);
          const int blocks = min(kBlocks, steps - kb);
          if (lead) mbar_arrive_expect_tx(&sm.full[st], blocks * bytes);
          const uint32_t fb = map_shared(&sm.full[st], 0);
          const int end = (walk.k0 + kb + blocks) * kBlockK;
          for (int k0 = (walk.k0 + kb) * kBlockK; k0 < end; k0 += kBlockK, as += kBlockBytes) {
            uint8_t* bs = as + kABytes;
            if (a.w_mn) {
              tma_load_3d_pair(as, &a.tw, fb, j, k0, walk.e);
              tma_load_3d_pair(as + 8192, &a.tw, fb, j + 64, k0, walk.e);
            } else {
              tma_load_3d_pair(as, &a.tw, fb, k0, j, walk.e);
            }
            // 128 rows, or those of 64, 32 and 16 that make up a half: no more than the products take.
#pragma unroll
            for (int b = 3, at = 0; b >= 0; --b) {
              if (half & (16 << b)) {
                tma_load_2d_pair(bs + at * 128, &a.tx[b], fb, k0, row + at);
                at += 16 << b;
              }
            }
          }
        }
        __syncwarp();
        next_stage(st, phase, a.stages);
      }
    }
    wait_copies(sm, n, a.stages, a.status);
  } else if (warp == 1 && lead) {
    const uint32_t s0 = (smem_u32(base) & 0x3FFFFu) >> 4;
    const uint64_t da = (a.w_mn ? sdesc_mn_sw128(0) : sdesc_k_sw128(0)) + s0;
    const uint64_t db = sdesc_k_sw128(0) + s0 + (kABytes >> 4);
    const uint32_t step_a = (a.w_mn ? 2048 : 32) >> 4;
    int it = 0, st = 0;
    uint32_t phase = 0, at = 0;  // at: the stage's offset in 16-byte units
    bool ok = true;
    for (; ok && walk.next(); ++it) {
      const uint32_t idesc = idesc_16bit(kBf16, a.w_mn, false, kFeatures, walk.cols);
      const int acc = it & 1, steps = walk.steps();
      if (!warp_pwait(&sm.tempty[acc], ((it >> 1) & 1) ^ 1, &sm.abort, a.status, 0x44000000u)) break;
      tc_fence_after();
      const uint32_t dt = tmem + (uint32_t)(acc * kRows);
      for (int kb = 0; kb < steps; kb += kBlocks) {
        if (!warp_pwait(&sm.full[st], phase, &sm.abort, a.status, 0x45000000u)) {
          ok = false;
          break;
        }
        tc_fence_after();
        if (elect_one()) {
#pragma unroll
          for (int k = 0; k < kBlockK / 16; ++k)
            tc_mma_pair(dt, da + at + k * step_a, db + at + k * (32 >> 4), idesc, (kb | k) != 0 ? 1u : 0u);
          if (kb + 1 < steps) {
            const uint32_t bt = at + (kBlockBytes >> 4);
#pragma unroll
            for (int k = 0; k < kBlockK / 16; ++k)
              tc_mma_pair(dt, da + bt + k * step_a, db + bt + k * (32 >> 4), idesc, 1u);
          }
          tc_commit_pair(&sm.empty[st], 0x3);
        }
        __syncwarp();
        next_stage(st, phase, a.stages);
        at = st == 0 ? 0 : at + (kBlocks * kBlockBytes >> 4);
      }
      if (ok && elect_one()) tc_commit_pair(&sm.tfull[acc], 0x3);
      __syncwarp();
    }
    wait_products(sm, a.status);
  } else if (warp >= 2) {
    // A warp has 32 features (its lane quarter of TMEM) and every other 32 rows of the tile. Turned
    // round in shared memory, four lanes store the 32 features of a row; what is added comes the same way
    // back (read by features, 2 bytes a lane, it took 450 us where this takes 422: dx of 128 experts of 256
    // rows, 2048 x 4096).
    const int q = warp & 3, half = (warp - 2) >> 2;
    const uint32_t tempty[2] = {map_shared(&sm.tempty[0], 0), map_shared(&sm.tempty[1], 0)};
    uint8_t* patch = patches + (warp - 2) * kPatchBytes;
    unsigned short* y = static_cast<unsigned short*>(a.y);
    const unsigned short* add = static_cast<const unsigned short*>(a.add);
    for (int it = 0; walk.next(); ++it) {
      const int acc = it & 1;
      const int f0 = walk.j0 + (int)crank * 128 + q * 32, nf = a.J - f0;
      const uint32_t src = tmem + ((uint32_t)(q * 32) << 16) + (uint32_t)(acc * kRows);
      const int chunks = (walk.rows + 31) / 32;
      const bool zero = walk.e >= a.E;
      int c = half;
      // What is added to 32 rows, as it is stored: four lanes a row. On its way before the sums are waited for.
      uint4 u[4];
      auto fetch = [&](int chunk) {
        const unsigned short* p = add + (long long)(walk.row0 + chunk * 32) * a.ld_add + f0 + (lane & 3) * 8;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int x = (lane >> 2) + 8 * i;
          u[i] = x < walk.rows - chunk * 32 && (lane & 3) * 8 < nf
                     ? __ldg(reinterpret_cast<const uint4*>(p + x * a.ld_add))
                     : make_uint4(0, 0, 0, 0);
        }
      };
      if (a.add != nullptr && c < chunks) fetch(c);
      if (!warp_pwait(&sm.tfull[acc], (it >> 1) & 1, &sm.abort, a.status, 0x46000000u)) break;
      tc_fence_after();
      do {
        uint32_t va[16], vb[16];  // the first 16 features and the others
        __syncwarp();  // the stores before may have parted it; the load wants it whole
        if (c < chunks) {
          tmem_ld_pieces(src + c * 32, va);
          tmem_ld_pieces(src + (16u << 16) + c * 32, vb);
          tmem_ld_wait();
        }
        if (c + 2 >= chunks) {  // the accumulator is read: it may be overwritten
          tc_fence_before();
          __syncwarp();
          if (lane == 0) arrive_read(tempty[acc]);
        }
        if (c < chunks && nf > 0) {
          const long long r0 = walk.row0 + c * 32;
          const int rows = min(32, walk.rows - c * 32);
          if (a.part != nullptr) {  // few rows: each thread its own sums, eight features together
            float* to = a.part + ((long long)walk.split * a.n + r0) * a.J + f0;
#pragma unroll
            for (int i = 0; i < 32; ++i) {
              const int f = (lane >> 2) + (i & 2 ? 8 : 0) + (i & 16), x = (i >> 2 & 3) * 8 + 2 * (lane & 3) + (i & 1);
              const uint32_t v = i < 16 ? va[i & 15] : vb[i & 15];
              if (x < rows && f < nf) to[(long long)x * a.J + f] = zero ? 0.f : __uint_as_float(v);
            }
            c += 2;
            continue;
          }
          __syncwarp();  // the patch's last readers
          if (a.add != nullptr) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
              *reinterpret_cast<uint4*>(patch + patch_at((lane >> 2) + 8 * i, lane & 3)) = u[i];
            if (c + 2 < chunks) fetch(c + 2);
            __syncwarp();
          }
          // Eight rows at a time, turned round as they are stored (element by element, 32 stores of 2 bytes,
          // a chunk took 1050 cycles).
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint32_t at = smem_u32(patch + patch_at(8 * i + (lane & 7), lane >> 3));
            uint32_t w[4] = {0, 0, 0, 0};
            if (a.add != nullptr) load_turned(at, w);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const uint32_t* v = (k < 2 ? va : vb) + 4 * i + 2 * (k & 1);
              float lo = zero ? 0.f : __uint_as_float(v[0]), hi = zero ? 0.f : __uint_as_float(v[1]);
              if (a.add != nullptr) {
                const float2 f = unpack2<T>(w[k]);
                lo += f.x;
                hi += f.y;
              }
              w[k] = pack2<T>(lo, hi);
            }
            store_turned(at, w);
          }
          __syncwarp();
          const int f = (lane & 3) * 8;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int x = (lane >> 2) + 8 * i;
            const uint4 o = *reinterpret_cast<const uint4*>(patch + patch_at(x, lane & 3));
            if (x < rows && f < nf) *reinterpret_cast<uint4*>(y + (r0 + x) * a.ld_y + f0 + f) = o;
          }
        }
        c += 2;
      } while (c < chunks);
    }
  }
  pair_teardown(tmem, warp);
}

// The parts' sums of every element, in their order, with what is added, rounded once.
template <typename T>
__global__ void __launch_bounds__(256) expert_join_kernel(const __grid_constant__ RowsArgs a) {
  wait_prior_grid();
  const long long per = a.J / 8, all = a.n * per;
  for (long long i = (long long)blockIdx.x * 256 + threadIdx.x; i < all; i += (long long)gridDim.x * 256) {
    const long long row = i / per, c = (i - row * per) * 8;
    float f[8];
    for (int s = 0; s < 1 << a.split_bits; ++s) {
      const float4* q = reinterpret_cast<const float4*>(a.part + ((long long)s * a.n + row) * a.J + c);
      const float4 u = q[0], v = q[1];
      const float w[8] = {u.x, u.y, u.z, u.w, v.x, v.y, v.z, v.w};
#pragma unroll
      for (int k = 0; k < 8; ++k) f[k] = s == 0 ? w[k] : f[k] + w[k];
    }
    if (a.add != nullptr) {
      float g[8];
      unpack<T>(__ldg(reinterpret_cast<const uint4*>(static_cast<const T*>(a.add) + row * a.ld_add + c)), g);
#pragma unroll
      for (int k = 0; k < 8; ++k) f[k] += g[k];
    }
    *reinterpret_cast<uint4*>(static_cast<T*>(a.y) + row * a.ld_y + c) = pack<T>(f);
  }
}

// ------------------------------------------------------------------- dW
struct WeightArgs {
  CUtensorMap ty, tx;  // rows of dy and of x
  CUtensorMap tw;      // dW, 32 rows of 64 bytes
  const int32_t* offsets;
  void* dw;                 // [E][N][K], rows ld apart, experts `stride`
  long long ld, stride;
  uint32_t* status;
  int n, E, N, K;
  int tiles_i, tiles_j, stages;
};

// The tensor cores' fp32 sums lose what lies below their last bit at every step, so their error grows with the
// number of rows: relative to dW's norm 3.4e-7 for 256 random rows, 9.4e-7 for 768, then 1.2e-9 a row (3.8e-5 for
// 32768). An fp32 dW therefore takes a tile's rows in parts, which are added to what is stored by copies that add
// (fp32, rounded to nearest, one after the other): 1.0e-6 up to 262144 rows, 1.2e-6 for 1048576, the parts'
// own roundings. (16384 rows, 2048 x 4096: 157 us in one part, 223 by parts of 1024, 255 by 768, 313 by 512.) In 16
// bits there is one part: the rounding of dW itself is 2.1e-4 of its norm in fp16 and 1.7e-3 in bf16, which
// the sum's error reaches at some 170000 rows of one expert in fp16 and at 1.4 million in bf16 (in all,
// 262144 rows in fp16 are off by 3.7e-4, 1048576 in bf16 by 2.1e-3).
constexpr int kPartRows = 768;

// The tiles of a pair: p, p + pairs, ... of the order expert, rows, columns of dW: the tiles in flight
// write whole rows. PART: rows of a sum that the tensor cores take at once; the parts of a tile come one after
// the other.
template <int PART>
struct WeightWalk {
  const WeightArgs& a;
  int per, local, step_e, step_local;  // tiles of an expert; the position is e * per + local
  int e, i0, j0, cols;      // the tile: expert, first row and column, columns: 256, or 128 at the right edge
  int start, count, steps;  // the expert's rows, or a part of them; blocks of 64 of them
  int left;                 // rows of the parts after it
  bool more;                // a part after the first

  __device__ __forceinline__ WeightWalk(const WeightArgs& args, int pair, int n)
      : a(args), per(a.tiles_i * a.tiles_j), i0(0), j0(0), cols(0), start(0), count(0), steps(0), left(0), more(false) {
    step_e = n / per;
    step_local = n - step_e * per;
    e = pair / per - step_e;
    local = pair - pair / per * per - step_local;
  }
  __device__ __forceinline__ void take() {
    left = max(count - PART, 0);
    count = min(count, PART);
    steps = (count + kBlockK - 1) / kBlockK;
  }
  __device__ __forceinline__ bool next() {
    more = left > 0;
    if (more) {
      start += count;
      count = left;
      take();
      return true;
    }
    e += step_e;
    local += step_local;
    if (local >= per) {
      local -= per;
      ++e;
    }
    if (e >= a.E) return false;
    const int ti = local / a.tiles_j;
    i0 = ti * 256;
    j0 = (local - ti * a.tiles_j) * 256;
    cols = a.K - j0 <= 128 ? 128 : 256;
    rows_of(a.offsets, e, a.E, a.n, &start, &count);
    take();
    return true;
  }
};

// dW[e] = sum over the rows of e of dy[r] x[r]^T: both operands lie row by row, so both go to the tensor cores with
// the sum outermost, 64 rows at a time. With few rows of many experts it is bound by what it writes, dW once
// (64 experts of 4 rows, 2048 x 4096: 195 us, 5.5 TB/s; 128 of 32: 375, 5.9; 5 of 64 with rows: 171, 6.3), with
// many by the products (16384 rows of one, 2048 x 4096: 154 us, 1.78 PFLOP/s). A pair's tile takes all rows
// of its expert, for an fp32 dW in parts (kPartRows). T: the operands' type; O: dW's, T or float.
template <typename T, typename O>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kWeightThreads, 1)
    expert_weights_kernel(const __grid_constant__ WeightArgs a) {
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  uint8_t* base = smem_raw + (((raw + 1023u) & ~1023u) - raw);
  uint8_t* patches = base + (size_t)a.stages * kBlockBytes;
  PairSmem& sm = *reinterpret_cast<PairSmem*>(patches + kWeightEpiWarps * kPatchBytes);
  constexpr bool kBf16 = std::is_same<T, __nv_bfloat16>::value;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t crank = cluster_ctarank();
  const bool lead = crank == 0;
  pair_setup(sm, a.stages, warp, 2, kWeightEpiWarps);
  const uint32_t tmem = sm.tmem;
  wait_prior_grid();
  WeightWalk<sizeof(O) == 4 ? kPartRows : INT32_MAX> walk(a, blockIdx.x >> 1, gridDim.x >> 1);

  if (warp == 0) {
    int n = 0, st = 0;
    uint32_t phase = 1;
    bool ok = true;
    while (ok && walk.next()) {
      const int half = walk.cols / 2, i = walk.i0 + (int)crank * 128, j = walk.j0 + (int)crank * half;
      const uint32_t bytes = kABytes + half * 128;
      for (int kb = 0; kb < walk.steps; ++kb, ++n) {
        if (!warp_pwait(&sm.empty[st], phase, &sm.abort, a.status, 0x51000000u)) {
          ok = false;
          break;
        }
        if (elect_one()) {
          uint8_t* as = base + (size_t)st * kBlockBytes;
          uint8_t* bs = as + kABytes;
          const int row = walk.start + kb * kBlockK;
          uint32_t bar;
          if (walk.count - kb * kBlockK < kBlockK) {  // the warps that clear the rest fill this stage
            mbar_arrive_expect_tx(&sm.last[st], bytes);
            bar = map_shared(&sm.last[st], crank);
          } else {
            if (lead) {
              mbar_arrive_expect_tx(&sm.full[st], 2 * bytes);
              mbar_arrive(&sm.full[st]);
            }
            bar = map_shared(&sm.full[st], 0);
          }
          tma_load_2d_pair(as, &a.ty, bar, i, row);
          tma_load_2d_pair(as + 8192, &a.ty, bar, i + 64, row);
          tma_load_2d_pair(bs, &a.tx, bar, j, row);
          if (half > 64) tma_load_2d_pair(bs + 8192, &a.tx, bar, j + 64, row);
        }
        __syncwarp();
        next_stage(st, phase, a.stages);
      }
    }
    wait_copies(sm, n, a.stages, a.status);
  } else if (warp == 1 && lead) {
    const uint32_t s0 = (smem_u32(base) & 0x3FFFFu) >> 4;
    const uint64_t da = sdesc_mn_sw128(0) + s0, db = da + (kABytes >> 4);
    int it = 0, st = 0;
    uint32_t phase = 0, at = 0;
    bool ok = true;
    while (ok && walk.next()) {
      if (walk.steps == 0) continue;  // zeros: the epilogue's alone
      const int acc = it & 1;
      if (!warp_pwait(&sm.tempty[acc], ((it >> 1) & 1) ^ 1, &sm.abort, a.status, 0x54000000u)) break;
      tc_fence_after();
      const uint32_t dt = tmem + (uint32_t)(acc * 256), idesc = idesc_16bit(kBf16, true, true, 256, walk.cols);
      for (int kb = 0; kb < walk.steps; ++kb) {
        if (!warp_pwait(&sm.full[st], phase, &sm.abort, a.status, 0x55000000u)) {
          ok = false;
          break;
        }
        tc_fence_after();
        if (elect_one()) {
#pragma unroll
          for (int k = 0; k < kBlockK / 16; ++k)
            tc_mma_pair(dt, da + at + k * (2048 >> 4), db + at + k * (2048 >> 4), idesc, (kb | k) != 0 ? 1u : 0u);
          tc_commit_pair(&sm.empty[st], 0x3);
        }
        __syncwarp();
        next_stage(st, phase, a.stages);
        at = st == 0 ? 0 : at + (kBlockBytes >> 4);
      }
      if (ok && elect_one()) tc_commit_pair(&sm.tfull[acc], 0x3);
      __syncwarp();
      ++it;
    }
    wait_products(sm, a.status);
  } else if (warp == 2 + kWeightEpiWarps) {
    // Clears the rows past the expert's last in this CTA's half of its last block: they are another
    // expert's (or what lies behind the rows), and a NaN there times zero would be one. A block is
    // 64 rows of 128 bytes for each 64 columns; the swizzle stays inside a row.
    int n = 0;
    uint32_t used = 0;  // bit i: the phase of last[i]
    while (walk.next()) {
      n += walk.steps;
      const int rows = walk.count - (walk.steps - 1) * kBlockK;
      if (walk.steps == 0 || rows == kBlockK) continue;
      const int st = (n - 1) % a.stages;
      if (!warp_pwait(&sm.last[st], (used >> st) & 1, &sm.abort, a.status, 0x57000000u)) break;
      used ^= 1u << st;
      uint8_t* at = base + (size_t)st * kBlockBytes;
      for (int o = rows * 128 + lane * 16; o < 8192; o += 512) {
#pragma unroll
        for (int b = 0; b < kBlockBytes / 8192; ++b)
          *reinterpret_cast<uint4*>(at + b * 8192 + o) = make_uint4(0, 0, 0, 0);
      }
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // the products read by the async proxy
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster(map_shared(&sm.full[st], 0));
    }
  } else if (warp >= 2) {
    constexpr int kColumns = 256 * 4 / kWeightEpiWarps;
    const int q = warp & 3, from = ((warp - 2) >> 2) * kColumns;  // TMEM lane quarter, first column
    const uint32_t tempty[2] = {map_shared(&sm.tempty[0], 0), map_shared(&sm.tempty[1], 0)};
    uint8_t* patch = patches + (warp - 2) * kPatchBytes;
    int it = 0;
    while (walk.next()) {
      const int i = walk.i0 + (int)crank * 128 + q * 32 + lane;
      O* to = static_cast<O*>(a.dw) + walk.e * a.stride + (long long)(i - lane) * a.ld;  // the warp's first row
      const int rows = a.N - (i - lane);
      if (walk.steps == 0) {  // an expert without rows
        constexpr int kLanes = kColumns * (int)sizeof(O) / 16;  // of a row
        const int j = walk.j0 + from + lane % kLanes * (16 / (int)sizeof(O));
#pragma unroll 4
        for (int r = lane / kLanes; r < 32; r += 32 / kLanes)
          if (r < rows && j < a.K) *reinterpret_cast<uint4*>(to + r * a.ld + j) = make_uint4(0, 0, 0, 0);
        continue;
      }
      const int acc = it & 1;
      if (!warp_pwait(&sm.tfull[acc], (it >> 1) & 1, &sm.abort, a.status, 0x56000000u)) break;
      ++it;
      tc_fence_after();
      if (walk.more && lane == 0) bulk_wait_all();  // what is added to has been written
      const uint32_t src = tmem + ((uint32_t)(q * 32) << 16) + (uint32_t)(acc * 256);
#pragma unroll 1
      for (int c = from; c < from + kColumns; c += 32) {
        uint32_t v[32];
        __syncwarp();
        tmem_ld32(src + c, v);
        tmem_ld_wait();
        if (c + 32 == from + kColumns) {  // the accumulator is read: it may be overwritten
          tc_fence_before();
          __syncwarp();
          if (lane == 0) arrive_read(tempty[acc]);
        }
        // 32 rows of 64 bytes by way of shared memory, from which a copy takes them (dW of 128 experts of 128
        // rows, 2048 x 4096: 441 us; stored by the lanes, four of them a row, 463; of 64 experts of 4 rows 197
        // and 232).
        constexpr int kPart = 64 / (int)sizeof(O);  // columns of 64 bytes
#pragma unroll
        for (int h = 0; h < 32; h += kPart) {
          uint32_t w[16];
#pragma unroll
          for (int x = 0; x < 16; ++x) {
            if constexpr (sizeof(O) == 4)
              w[x] = v[h + x];
            else
              w[x] = pack2<T>(__uint_as_float(v[2 * x]), __uint_as_float(v[2 * x + 1]));
          }
          if (lane == 0) bulk_wait_read<0>();  // the patch's last copy
          __syncwarp();
#pragma unroll
          for (int x = 0; x < 4; ++x)
            *reinterpret_cast<uint4*>(patch + patch_at(lane, x)) =
                make_uint4(w[4 * x], w[4 * x + 1], w[4 * x + 2], w[4 * x + 3]);
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          __syncwarp();
          const int j = walk.j0 + c + h;
          if (rows > 0 && j < a.K && lane == 0) {
            if (sizeof(O) == 4 && walk.more)
              tma_add_3d(&a.tw, patch, j, i, walk.e);
            else
              tma_store_3d(&a.tw, patch, j, i, walk.e);
            bulk_commit();
          }
        }
      }
    }
    if (lane == 0) bulk_wait_all();
    __syncwarp();
  }
  pair_teardown(tmem, warp);
}

// ------------------------------------------------------------------- host side
// Map of a matrix of 16-bit elements, [rows][cols] or [experts][rows][cols]: boxes of box_rows x 64
// columns, 128-byte swizzle, zeros outside.
bool make_map(CUtensorMap* m, const void* p, bool bf16, long long experts, long long rows, long long cols,
              long long ld, long long stride, int box_rows) {
  const auto encode = tensor_map_encoder();
  if (encode == nullptr) return false;
  if (rows == 1) ld = cols;  // the stride of a single row, or expert, is never used
  if (experts == 1) stride = rows * ld;
  cuuint64_t dims[3] = {(cuuint64_t)cols, (cuuint64_t)rows, (cuuint64_t)experts};
  cuuint64_t strides[2] = {(cuuint64_t)ld * 2, (cuuint64_t)stride * 2};
  cuuint32_t box[3] = {(cuuint32_t)kBlockK, (cuuint32_t)box_rows, 1};
  cuuint32_t estr[3] = {1, 1, 1};
  return encode(m, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, experts > 0 ? 3 : 2,
                const_cast<void*>(p), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

constexpr long long kMaxSize = INT32_MAX / 2;

int check_experts(const moe_expert_linear_args* p) {
  if (p == nullptr) return MOE_ERR_ARG;
  if (p->dtype != MOE_BF16 && p->dtype != MOE_FP16) return MOE_ERR_ARG;
  if (p->n < 0 || p->n > kMaxSize || p->N < 8 || p->N > kMaxSize || p->K < 8 || p->K > kMaxSize || p->N % 8 != 0 ||
      p->K % 8 != 0 || p->E < 1 || p->E > kMaxExperts || p->offsets == nullptr || !aligned_to(p->offsets, 4))
    return MOE_ERR_ARG;
  return MOE_OK;
}
// Rows on 16 bytes.
bool check_matrix(const void* q, long long ld, long long rows, long long cols) {
  return q != nullptr && aligned_to(q, 16) && (rows <= 1 || (ld >= cols && ld % 8 == 0 && ld <= INT32_MAX));
}
bool check_weights(const void* q, long long ld, long long stride, const moe_expert_linear_args* p) {
  return check_matrix(q, ld, p->N, p->K) &&
         (p->E == 1 || (stride % 8 == 0 && stride >= (p->N - 1) * ld + p->K && stride <= 1LL << 38));
}
int launched(cudaError_t e) {
  if (e == cudaSuccess) return MOE_OK;
  cudaGetLastError();
  return MOE_ERR_CUDA;
}
size_t smem_bytes(size_t stages, size_t more) { return 1024 + stages + more + sizeof(PairSmem); }
// Stages of `bytes` that fit beside `more`.
int stages_for(size_t bytes, size_t more) {
  return std::min<int>(kMaxStages, (int)((kSmemMax - smem_bytes(0, more)) / bytes));
}

template <auto kKernel, typename A>
int launch_pairs(unsigned pairs, int threads, size_t smem, cudaStream_t s, const A& a) {
  static std::atomic<uint64_t> ready{0};
  cudaError_t e = allow_smem(reinterpret_cast<const void*>(kKernel), &ready);
  if (e == cudaSuccess) e = launch_behind(kKernel, dim3(2 * pairs), dim3((unsigned)threads), smem, s, a);
  return launched(e);
}

// Map of dW for stores: boxes of 32 rows of 64 bytes, whose 64-byte swizzle is that of the patches.
bool make_store_map(CUtensorMap* m, const moe_expert_linear_args* p) {
  const auto encode = tensor_map_encoder();
  if (encode == nullptr) return false;
  const cuuint64_t b = (cuuint64_t)type_bytes(p->dwtype);
  const long long ld = p->N == 1 ? p->K : p->ld_dw, stride = p->E == 1 ? p->N * ld : p->stride_dw;
  cuuint64_t dims[3] = {(cuuint64_t)p->K, (cuuint64_t)p->N, (cuuint64_t)p->E};
  cuuint64_t strides[2] = {(cuuint64_t)ld * b, (cuuint64_t)stride * b};
  cuuint32_t box[3] = {(cuuint32_t)(64 / b), 32, 1};
  cuuint32_t estr[3] = {1, 1, 1};
  const CUtensorMapDataType t = p->dwtype == MOE_FP32   ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
                                : p->dwtype == MOE_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                                        : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
  return encode(m, t, 3, p->dw, dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_64B,
                CU_TENSOR_MAP_L2_PROMOTION_NONE, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// How many pairs share a tile's sum (as a power of two), where its tiles leave half of 76 pairs idle or more and each
// gets eight blocks of 64 at least. Two rows of 256 features, a sum of 7168, eight parts: 9.2 us where one pair a
// tile takes 24; of 512 features and 2048, four parts: 7.6 and 10; eight rows of 1024 and 7168, two: 26 and 31.
// Sums below 32 blocks are left alone: the launch that joins the parts takes the 2 us that it saves.
int split_bits(long long n, long long J, long long sum, int E) {
  constexpr int kPairs = 76;
  const long long most = n / kRows + std::min<long long>(E + 1, n), tiles = most * ((J + kFeatures - 1) / kFeatures);
  const long long nk = (sum + kBlockK - 1) / kBlockK;
  int bits = 0;
  while (bits < 3 && nk >> (bits + 1) >= 8 && (tiles << (bits + 1)) <= kPairs) ++bits;
  return nk >= 32 ? bits : 0;
}

int check_parts(const moe_expert_linear_args* p, long long features, long long sum, const void* workspace,
                size_t bytes) {
  const size_t need = moe_expert_linear_workspace(p->n, features, sum, p->E);
  if (need > 0 && (workspace == nullptr || !aligned_to(workspace, 16))) return MOE_ERR_ARG;
  return bytes < need ? MOE_ERR_WORKSPACE : MOE_OK;
}

// y of the forward pass, or dx: `w_mn` takes W^T.
int rows_product(const moe_expert_linear_args* p, const void* x, long long ld_x, bool w_mn, const void* add,
                 long long ld_add, void* y, long long ld_y, int sms, void* workspace, cudaStream_t s) {
  RowsArgs a{};
  const bool bf16 = p->dtype == MOE_BF16;
  a.w_mn = w_mn;
  a.n = (int)p->n;
  a.E = p->E;
  a.J = (int)(w_mn ? p->K : p->N);
  const long long sum = w_mn ? p->N : p->K;
  a.nk = (int)((sum + kBlockK - 1) / kBlockK);
  a.split_bits = split_bits(p->n, a.J, sum, p->E);
  a.tiles_j = (a.J + kFeatures - 1) / kFeatures << a.split_bits;
  if (a.split_bits > 0) a.part = static_cast<float*>(workspace);
  a.offsets = p->offsets;
  a.y = y;
  a.ld_y = ld_y;
  a.add = add;
  a.ld_add = ld_add;
  a.status = ops_status();
  if (a.status == nullptr || !make_map(&a.tw, p->w, bf16, p->E, p->N, p->K, p->ld_w, p->stride_w, w_mn ? 64 : 128))
    return MOE_ERR_CUDA;
  for (int b = 0; b < 4; ++b)
    if (!make_map(&a.tx[b], x, bf16, 0, p->n, sum, ld_x, 0, 16 << b)) return MOE_ERR_CUDA;
  // Tiles of rows: one for every 256 and one more for each entry of the table at most.
  a.most = (int)(p->n / kRows + std::min<long long>(p->E + 2, p->n));
  const long long tiles = (long long)a.most * a.tiles_j;
  if (tiles > INT32_MAX / 2) return MOE_ERR_UNSUPPORTED;
  const size_t more = kEpiWarps * kPatchBytes + table_bytes(a.E);
  constexpr size_t kStage = kBlocks * kBlockBytes;
  a.stages = stages_for(kStage, more);
  const unsigned pairs = (unsigned)std::min<long long>(sms / 2, tiles);
  const size_t smem = smem_bytes(a.stages * kStage, more);
  const int rc = bf16 ? launch_pairs<expert_rows_product_kernel<__nv_bfloat16>>(pairs, kThreads, smem, s, a)
                      : launch_pairs<expert_rows_product_kernel<__half>>(pairs, kThreads, smem, s, a);
  if (rc != MOE_OK || a.part == nullptr) return rc;
  const dim3 grid((unsigned)std::min<long long>((p->n * (a.J / 8) + 255) / 256, 8 * sms));
  return launched(bf16 ? launch_behind(expert_join_kernel<__nv_bfloat16>, grid, dim3(256), 0, s, a)
                       : launch_behind(expert_join_kernel<__half>, grid, dim3(256), 0, s, a));
}

int weights_product(const moe_expert_linear_args* p, int sms, cudaStream_t s) {
  WeightArgs a{};
  const bool bf16 = p->dtype == MOE_BF16;
  if (!make_map(&a.ty, p->dy, bf16, 0, p->n, p->N, p->ld_dy, 0, kBlockK) ||
      !make_map(&a.tx, p->x, bf16, 0, p->n, p->K, p->ld_x, 0, kBlockK) || !make_store_map(&a.tw, p))
    return MOE_ERR_CUDA;
  a.offsets = p->offsets;
  a.dw = p->dw;
  a.ld = p->ld_dw;
  a.stride = p->stride_dw;
  a.status = ops_status();
  if (a.status == nullptr) return MOE_ERR_CUDA;
  a.n = (int)p->n;
  a.E = p->E;
  a.N = (int)p->N;
  a.K = (int)p->K;
  a.tiles_i = (a.N + 255) / 256;
  a.tiles_j = (a.K + 255) / 256;
  const long long tiles = (long long)a.tiles_i * a.tiles_j * a.E;
  if (tiles > INT32_MAX / 2) return MOE_ERR_UNSUPPORTED;
  constexpr size_t kMore = kWeightEpiWarps * kPatchBytes;
  a.stages = stages_for(kBlockBytes, kMore);
  const unsigned pairs = (unsigned)std::min<long long>(sms / 2, tiles);
  const size_t smem = smem_bytes((size_t)a.stages * kBlockBytes, kMore);
  if (p->dwtype == MOE_FP32)
    return bf16 ? launch_pairs<expert_weights_kernel<__nv_bfloat16, float>>(pairs, kWeightThreads, smem, s, a)
                : launch_pairs<expert_weights_kernel<__half, float>>(pairs, kWeightThreads, smem, s, a);
  return bf16 ? launch_pairs<expert_weights_kernel<__nv_bfloat16, __nv_bfloat16>>(pairs, kWeightThreads, smem, s, a)
              : launch_pairs<expert_weights_kernel<__half, __half>>(pairs, kWeightThreads, smem, s, a);
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

size_t moe_expert_linear_workspace(long long n, long long features, long long sum, int E) {
  if (n < 1 || features < 1 || sum < 1 || E < 1) return 0;
  const int bits = split_bits(n, features, sum, E);
  return bits == 0 ? 0 : ((size_t)n * features * sizeof(float)) << bits;
}

int moe_expert_linear(const moe_expert_linear_args* p, void* workspace, size_t workspace_bytes, moe_stream_t stream) {
  int rc = check_experts(p);
  if (rc != MOE_OK) return rc;
  if (p->n == 0) return MOE_OK;
  if (!check_matrix(p->x, p->ld_x, p->n, p->K) || !check_weights(p->w, p->ld_w, p->stride_w, p) ||
      !check_matrix(p->y, p->ld_y, p->n, p->N))
    return MOE_ERR_ARG;
  rc = check_parts(p, p->N, p->K, workspace, workspace_bytes);
  if (rc != MOE_OK) return rc;
  int sms = 0;
  rc = ops_device(&sms);
  if (rc != MOE_OK) return rc;
  return rows_product(p, p->x, p->ld_x, false, nullptr, 0, p->y, p->ld_y, sms, workspace,
                      reinterpret_cast<cudaStream_t>(stream));
}

int moe_expert_linear_backward(const moe_expert_linear_args* p, void* workspace, size_t workspace_bytes,
                               moe_stream_t stream) {
  int rc = check_experts(p);
  if (rc != MOE_OK) return rc;
  if (p->dwtype != p->dtype && p->dwtype != MOE_FP32) return MOE_ERR_ARG;
  if (p->dw != nullptr && !check_weights(p->dw, p->ld_dw, p->stride_dw, p)) return MOE_ERR_ARG;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  int sms = 0;
  if (p->n == 0) {  // no rows: the weights' gradients are zero
    if (p->dw == nullptr) return MOE_OK;
    rc = ops_device(&sms);
    if (rc != MOE_OK) return rc;
    const size_t b = (size_t)type_bytes(p->dwtype), row = (size_t)p->K * b;
    for (int e = 0; e < p->E; ++e)
      if (cudaMemset2DAsync(static_cast<char*>(p->dw) + (size_t)e * p->stride_dw * b,
                            p->N > 1 ? (size_t)p->ld_dw * b : row, 0, row, (size_t)p->N, s) != cudaSuccess)
        return launched(cudaErrorUnknown);
    return MOE_OK;
  }
  if (!check_matrix(p->dy, p->ld_dy, p->n, p->N) ||
      (p->dx != nullptr && (!check_matrix(p->dx, p->ld_dx, p->n, p->K) ||
                            !check_weights(p->w, p->ld_w, p->stride_w, p) ||
                            (p->add != nullptr && !check_matrix(p->add, p->ld_add, p->n, p->K)))) ||
      (p->dw != nullptr && !check_matrix(p->x, p->ld_x, p->n, p->K)))
    return MOE_ERR_ARG;
  if (p->dx != nullptr && (rc = check_parts(p, p->K, p->N, workspace, workspace_bytes)) != MOE_OK) return rc;
  rc = ops_device(&sms);
  if (rc != MOE_OK) return rc;
  if (p->dx != nullptr)
    rc = rows_product(p, p->dy, p->ld_dy, true, p->add, p->ld_add, p->dx, p->ld_dx, sms, workspace, s);
  if (rc == MOE_OK && p->dw != nullptr) rc = weights_product(p, sms, s);
  return rc;
}

}  // extern "C"
