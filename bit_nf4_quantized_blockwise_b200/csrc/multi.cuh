// multi.cuh - the linear layer with many adapters beside one frozen weight:
// token i uses adapter a_i of a bank (or none),
//   Y_i  = X_i W' + s[a_i] T_i L2[a_i],         T_i = X_i L1[a_i]
//   dX_i = dY_i W'^T + s[a_i] U_i L1[a_i]^T,    U_i = dY_i L2[a_i]^T
//   dL1[a] = s[a] sum_{a_i = a} X_i^T U_i,  dL2[a] = s[a] sum_{a_i = a} T_i^T dY_i
// (the LoRA equation of the walkthrough's background section and its training
// step 5, with the factors chosen per token).
//
// adapter_plan_kernel sorts the tokens of a batch into groups of one adapter,
// in the order of first appearance, so that a batch whose adapters are already
// contiguous (whole requests one after the other) keeps its order and nothing
// has to be moved.  Everything below works on sorted rows.
//
// The rank-r product of a group is appended to the K loop of the W' product, as
// in the one-adapter GEMM, but per 256-row tile and only for the groups that
// have rows in it: a *slot* is one (tile, group) pair and holds the group's
// 256 x rp rows of s T as bf16 parts (hi, the rounding of what is left, and
// again), with zeros in the rows of other groups.  A batch has at most
// tiles + groups slots.
//
// Zero rows keep the groups apart only while the factors are finite: 0 times an
// infinity or a NaN of another group's adapter (or of another token, in the
// sums over tokens) is NaN.  And a value in parts, hi inf + mid inf, is NaN where the
// value itself times inf is not.  Every element that comes out non-finite is
// therefore computed once more from its own row and adapter alone, in fp32 and
// with whole values; a finite batch never gets there.
//
// Times in these comments are of calls in a loop over two or three sets of inputs at
// the step that they describe, unless they say cold; a call with a cold L2 takes 2 to
// 15 % longer.
#pragma once

#include "qlora.h"

#include "common.cuh"
#include "gemm.cuh"
#include "pairgemm.cuh"

namespace qlora {

// ====================================================================== the plan of a batch

constexpr int MP_THREADS = 1024;
constexpr int MP_WARPS = MP_THREADS / 32;
constexpr int MP_SLOT_ROWS = 256;  // rows of a slot: those of a pair tile
constexpr int MP_TILE = 64;        // rows of a tile of the rank-r products

struct PlanHead {
  int groups;    // adapters with tokens
  int in_order;  // the sorted order is the batch's own
  int slots;
  int tiles;     // 64-row tiles of the groups
};

// A group: its rows are the sorted positions start .. end - 1.
struct PlanGroup {
  int adapter, start, end;
  int slot0;  // its first slot
};
struct PlanSlot {
  int adapter, start, end;  // of the group
  int tile;                 // 256-row tile
};
struct PlanTile {
  int adapter, row0, rows;  // up to 64 rows of a group
  int group;
};

// Arrays of a plan (device); lengths in brackets, G = min(n, M).  A kernel gets
// what it needs of a group, slot or tile with one 16-byte load: chains of
// dependent loads at the start of every block are most of what a small batch
// costs.
struct PlanView {
  PlanHead* head;
  int* perm;         // [M] row of the batch at sorted position p
  int* owner;        // [M] adapter of row i of the batch, -1: none
  PlanGroup* groups; // [G]
  int* adp_group;    // [n] group of an adapter, -1: no tokens
  PlanSlot* slots;   // [slots]
  int* tile_slot0;   // [tiles + 1] first slot of a 256-row tile
  PlanTile* tiles;   // [64-row tiles]
  int* counts;       // scratch: [32][n + 1], then [n + 1] each of first, total, start
  int M, n;
};

template <typename T>
__device__ __forceinline__ T plan_load(const T* p) {
  static_assert(sizeof(T) == 16, "one 16-byte load");
  const int4 x = __ldg(reinterpret_cast<const int4*>(p));
  return *reinterpret_cast<const T*>(&x);
}

// Sum over the block's threads before this one, and the total (x, y apart).
__device__ __forceinline__ int2 block_scan(int2 v, int2 (&sh)[MP_WARPS], int2& total) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int2 s = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int x = __shfl_up_sync(0xFFFFFFFFu, s.x, o), y = __shfl_up_sync(0xFFFFFFFFu, s.y, o);
    if (lane >= o) s.x += x, s.y += y;
  }
  __syncthreads();  // sh of the scan before this one has been read
  if (lane == 31) sh[warp] = s;
  __syncthreads();
  int2 before = make_int2(0, 0);
  total = make_int2(0, 0);
  for (int w = 0; w < MP_WARPS; ++w) {
    if (w < warp) before.x += sh[w].x, before.y += sh[w].y;
    total.x += sh[w].x, total.y += sh[w].y;
  }
  return make_int2(before.x + s.x - v.x, before.y + s.y - v.y);
}

// A stable counting sort by adapter in one block: each warp counts a contiguous
// part of the tokens (equal adapters of a 32-token step by match), the counts
// are summed over the warps, the groups are placed by a scan over the tokens
// that are the first of their adapter, and each warp writes its part.  Once
// per batch, for all layers; adapters outside 0 .. n - 1 mean none.
__global__ void __launch_bounds__(MP_THREADS) adapter_plan_kernel(const int* __restrict__ adapter, const PlanView v) {
  __shared__ int2 sh[MP_WARPS];
  __shared__ int moved;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int M = v.M, n = v.n, keys = n + 1;  // key n: no adapter
  int* first = v.counts + MP_WARPS * keys;
  int* total = first + keys;
  int* start = total + keys;
  for (int i = threadIdx.x; i < MP_WARPS * keys; i += MP_THREADS) v.counts[i] = 0;
  for (int i = threadIdx.x; i < keys; i += MP_THREADS) first[i] = 0x7FFFFFFF;
  for (int i = threadIdx.x; i < n; i += MP_THREADS) v.adp_group[i] = -1;
  if (threadIdx.x == 0) moved = 0;
  __syncthreads();
  const int part = ((M + MP_THREADS - 1) / MP_THREADS) * 32;  // tokens of a warp
  const int64_t w0 = static_cast<int64_t>(part) * warp;
  const int64_t w1 = w0 + part < M ? w0 + part : M;
  int* mine = v.counts + warp * keys;
  for (int64_t b = w0; b < w1; b += 32) {
    const int i = static_cast<int>(b) + lane;
    const bool in = i < w1;
    int key = -1;
    if (in) {
      const int a = adapter[i];
      key = a >= 0 && a < n ? a : n;
      v.owner[i] = key < n ? key : -1;
    }
    const unsigned same = __match_any_sync(0xFFFFFFFFu, key);
    if (in && lane == __ffs(same) - 1) {
      mine[key] += __popc(same);
      atomicMin(first + key, i);
    }
    __syncwarp();
  }
  __syncthreads();
  for (int key = threadIdx.x; key < keys; key += MP_THREADS) {
    int run = 0;
    for (int w = 0; w < MP_WARPS; ++w) {
      const int c = v.counts[w * keys + key];
      v.counts[w * keys + key] = run;
      run += c;
    }
    total[key] = run;
  }
  __syncthreads();
  int2 carry = make_int2(0, 0);  // groups and rows placed so far
  for (int64_t b = 0; b < M; b += MP_THREADS) {
    const int64_t i = b + threadIdx.x;
    int key = -1;
    if (i < M) {
      const int a = v.owner[i];
      key = a < 0 ? n : a;
      if (first[key] != i) key = -1;
    }
    int2 sum;
    const int2 at = block_scan(make_int2(key >= 0 && key < n ? 1 : 0, key >= 0 ? total[key] : 0), sh, sum);
    if (key >= 0) {
      start[key] = carry.y + at.y;
      if (key < n) {
        const int g = carry.x + at.x;
        v.groups[g] = {key, start[key], start[key] + total[key], 0};
        v.adp_group[key] = g;
      }
    }
    carry.x += sum.x, carry.y += sum.y;
  }
  const int groups = carry.x;
  __syncthreads();
  for (int64_t b = w0; b < w1; b += 32) {
    const int i = static_cast<int>(b) + lane;
    const bool in = i < w1;
    int key = -1;
    if (in) {
      const int a = v.owner[i];
      key = a < 0 ? n : a;
    }
    const unsigned same = __match_any_sync(0xFFFFFFFFu, key);
    if (in) {
      const int p = start[key] + mine[key] + __popc(same & ((1u << lane) - 1u));
      v.perm[p] = i;
      if (p != i) moved = 1;
    }
    __syncwarp();
    if (in && lane == __ffs(same) - 1) mine[key] += __popc(same);
    __syncwarp();
  }
  __syncthreads();
  carry = make_int2(0, 0);  // slots and 64-row tiles
  for (int b = 0; b < groups; b += MP_THREADS) {
    const int g = b + threadIdx.x;
    int t0 = 0;
    PlanGroup pg{};
    int2 c = make_int2(0, 0);
    if (g < groups) {
      pg = v.groups[g];
      t0 = pg.start / MP_SLOT_ROWS;
      c.x = (pg.end - 1) / MP_SLOT_ROWS - t0 + 1;
      c.y = (pg.end - pg.start + MP_TILE - 1) / MP_TILE;
    }
    int2 sum;
    const int2 at = block_scan(c, sh, sum);
    if (g < groups) {
      const int s0 = carry.x + at.x, y0 = carry.y + at.y;
      v.groups[g].slot0 = s0;
      for (int k = 0; k < c.x; ++k) v.slots[s0 + k] = {pg.adapter, pg.start, pg.end, t0 + k};
      for (int k = 0; k < c.y; ++k)
        v.tiles[y0 + k] = {pg.adapter, pg.start + MP_TILE * k, min(MP_TILE, pg.end - pg.start - MP_TILE * k), g};
    }
    carry.x += sum.x, carry.y += sum.y;
  }
  __syncthreads();
  const int tiles = (M + MP_SLOT_ROWS - 1) / MP_SLOT_ROWS;
  for (int t = threadIdx.x; t <= tiles; t += MP_THREADS) {
    int lo = 0, hi = carry.x;  // the first slot whose tile is t or later
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (v.slots[mid].tile < t)
        lo = mid + 1;
      else
        hi = mid;
    }
    v.tile_slot0[t] = lo;
  }
  if (threadIdx.x == 0) *v.head = {groups, moved ? 0 : 1, carry.x, carry.y};
}

// ====================================================================== rank-r products of the groups

// D[p][j] = sum_k A[perm[p]][k] B[a][..] for 64 rows of one group and one part of
// K: T = X L1 (kKN: the factor is [K][r]) and U = dY L2^T ([r][K]).  Each part
// stores its own fp32 sums (pack adds them in order).  mma.sync and not
// tcgen05: its 16-row granularity lets a group of one token cost one fragment
// row instead of 128, and rows are gathered by cp.async wherever they lie.  The
// product reads its rows once at 2 r operations a value, so memory bounds it for
// r up to 64.  4-deep ring, 64 of K a stage; rows of 144 and 2 RP + 16 bytes keep
// ldmatrix free of bank conflicts.  Tiles of 128 rows (32 a warp) halve the
// reads of B from shared memory but leave 8 warps an SM: not faster at 4096 x
// 4096 (16 us both), slower for small groups (333 tokens: 18 us for 11).
// Ranks above 128 are further blocks (blockIdx.z).
// The tensor core cuts its running sum to fp32 at every step, so after every
// MS_CHAIN stages the sums are added to others in registers: without this the
// cut is what dL1's error against 64 bits consists of (5.8e-6 of dL1's norm at K =
// 13824, 1.2e-6 with it; an fp32 product's is 1.3e-6).
constexpr int MS_THREADS = 128;
constexpr int MS_K = 64;
constexpr int MS_PITCH = MS_K * 2 + 16;
constexpr int MS_CHAIN = 4;       // stages
constexpr int MS_MAX_RP = 128;    // ranks of a block
template <int RP, bool kKN>
constexpr int ms_b_pitch() {
  return kKN ? RP * 2 + 16 : MS_PITCH;
}
template <int RP, bool kKN>
constexpr int ms_stage_bytes() {
  return MP_TILE * MS_PITCH + (kKN ? MS_K : RP) * ms_b_pitch<RP, kKN>();
}
template <int RP>
constexpr int ms_stages() {
  return RP <= 64 ? 4 : 3;
}

// Sorted copies of the rows of X (and dY), for batches that are not in the groups' order: further
// blocks of the rank-r product's grid, which gathers its own rows and is bound by latency.  As a kernel
// before it they were one launch more for every batch, and took 1084 us a call for 1065 (8190 shuffled
// tokens, 5120 x 13824, backward); copied by the blocks' threads instead of bulk copies 1107.
constexpr int MC_PER_SM = 2;  // such blocks
struct SortParams {
  const uint4* src[2];
  uint4* dst[2];
  int vecs[2];  // 16-byte vectors of a row (0: none)
  int blocks;   // of each split
};

struct ShrinkParams {
  const uint16_t* A;   // [M][K]
  const uint16_t* B;   // bank
  int64_t b_stride;    // elements between two adapters
  int64_t ldb;
  int K, r;
  int k_per_split;     // a multiple of 64
  float* P;            // [splits][M][r]
  float* zero;         // also zeroed by the grid: the accumulator of the decode kernel, or null
  int64_t zero_len;    // a multiple of 4
  SortParams sort;
};

// Block `block` of `blocks` copies rows through a ring of bulk copies, by one thread.
constexpr int MC_SLOTS = 4;
constexpr int MC_BYTES = 10240;  // of a slot; the ring fits the shared memory of every rank
__device__ __forceinline__ void sort_rows(const SortParams& p, const PlanView& v, int block, int blocks, uint8_t* ring) {
  uint64_t* full = reinterpret_cast<uint64_t*>(ring + MC_SLOTS * MC_BYTES);
  for (int s = 0; s < MC_SLOTS; ++s) mbar_init(&full[s], 1);
  fence_mbar_init();
  struct Piece {  // the next piece to load, or to store
    int64_t at;
    int side, off;
  };
  auto bytes = [&](int side) { return 16 * (side ? p.vecs[1] : p.vecs[0]); };
  auto src = [&](int side) { return reinterpret_cast<const uint8_t*>(side ? p.src[1] : p.src[0]); };
  auto dst = [&](int side) { return reinterpret_cast<uint8_t*>(side ? p.dst[1] : p.dst[0]); };
  auto next = [&](Piece& x) {
    x.off += MC_BYTES;
    if (x.off < bytes(x.side)) return;
    x.off = 0;
    if (x.side == 0 && bytes(1) > 0) {
      x.side = 1;
    } else {
      x.side = 0;
      x.at += blocks;
    }
  };
  Piece in{block, 0, 0}, out = in;
  int n_in = 0, n_out = 0;
  int64_t from = block < v.M ? __ldg(v.perm + block) : 0, ahead = block + blocks < v.M ? __ldg(v.perm + block + blocks) : 0;
  auto load = [&]() {
    if (in.at >= v.M) return;
    const int s = n_in++ % MC_SLOTS;
    const uint32_t len = static_cast<uint32_t>(min(MC_BYTES, bytes(in.side) - in.off));
    mbar_arrive_expect_tx(&full[s], len);
    bulk_load(ring + s * MC_BYTES, src(in.side) + from * bytes(in.side) + in.off, len, &full[s]);
    const int64_t row = in.at;
    next(in);
    if (in.at != row) {
      from = ahead;
      if (in.at + blocks < v.M) ahead = __ldg(v.perm + in.at + blocks);
    }
  };
  for (int s = 0; s < MC_SLOTS - 1; ++s) load();
  while (n_out < n_in) {
    const int s = n_out % MC_SLOTS;
    if (!mbar_wait(&full[s], (n_out / MC_SLOTS) & 1)) break;
    ++n_out;
    const uint32_t len = static_cast<uint32_t>(min(MC_BYTES, bytes(out.side) - out.off));
    asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(
                     dst(out.side) + out.at * bytes(out.side) + out.off),
                 "r"(smem_u32(ring + s * MC_BYTES)), "r"(len)
                 : "memory");
    asm volatile("cp.async.bulk.commit_group;" ::: "memory");
    next(out);
    asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory");  // the slot before this one has been read
    load();
  }
  for (; n_out < n_in; ++n_out) mbar_wait(&full[n_out % MC_SLOTS], (n_out / MC_SLOTS) & 1);  // after a wait that gave up
  asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool valid) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(valid ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr));
}
__device__ __forceinline__ void ldsm4_t(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr));
}

template <int RP, bool kKN>
__global__ void __launch_bounds__(MS_THREADS, RP <= 64 ? 3 : 2)
    multi_shrink_kernel(const __grid_constant__ ShrinkParams p, const __grid_constant__ PlanView v) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  constexpr int kStages = ms_stages<RP>();
  constexpr int kStage = ms_stage_bytes<RP, kKN>();
  constexpr int kBPitch = ms_b_pitch<RP, kKN>();
  static_assert(kStages * kStage >= MC_SLOTS * (MC_BYTES + 8), "the copies' ring");
  pdl_launch_dependents();
  if (p.zero != nullptr)
    for (int64_t q = (static_cast<int64_t>(blockIdx.y) * gridDim.x + blockIdx.x) * MS_THREADS + threadIdx.x;
         q < p.zero_len / 4; q += static_cast<int64_t>(gridDim.x) * gridDim.y * MS_THREADS)
      reinterpret_cast<float4*>(p.zero)[q] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  const int tile_blocks = static_cast<int>(gridDim.x) - p.sort.blocks;
  if (static_cast<int>(blockIdx.x) >= tile_blocks) {
    if (blockIdx.z == 0 && threadIdx.x == 0 && !__ldg(&v.head->in_order))
      sort_rows(p.sort, v, static_cast<int>(blockIdx.y) * p.sort.blocks + static_cast<int>(blockIdx.x) - tile_blocks,
                p.sort.blocks * static_cast<int>(gridDim.y), smem_raw);
    pdl_wait();
    return;
  }
  const int n_tiles = __ldg(&v.head->tiles);
  const PlanTile tile = plan_load(v.tiles + blockIdx.x);  // allocated for every block; garbage past n_tiles
  if (static_cast<int>(blockIdx.x) >= n_tiles) {
    pdl_wait();
    return;
  }
  const int j0 = static_cast<int>(blockIdx.z) * MS_MAX_RP;
  const int ranks = min(RP, p.r - j0);
  const uint16_t* B = p.B + static_cast<int64_t>(tile.adapter) * p.b_stride + (kKN ? j0 : j0 * p.ldb);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int k0 = blockIdx.y * p.k_per_split;
  const int k1 = min(p.K, k0 + p.k_per_split);
  const int steps = (k1 - k0) / MS_K;
  const uint32_t base = smem_u32(smem_raw);
  // this thread's rows of the A tile: 16 i + tid / 8, 16-byte column tid % 8
  const int mine = threadIdx.x >> 3;
  const uint16_t* arow[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int rr = 16 * i + mine;
    arow[i] = p.A + static_cast<int64_t>(__ldg(v.perm + tile.row0 + (rr < tile.rows ? rr : 0))) * p.K + 8 * (threadIdx.x & 7);
  }
  auto load = [&](int s) {
    if (s < steps) {
      const uint32_t st = base + (s % kStages) * kStage;
      const int k = k0 + s * MS_K;
      const uint32_t sb = st + MP_TILE * MS_PITCH;
      if constexpr (kKN) {
        constexpr int kVec = RP / 8;
#pragma unroll
        for (int q = threadIdx.x; q < MS_K * kVec; q += MS_THREADS) {
          const int kk = q / kVec, c = q % kVec;
          const bool ok = 8 * c < ranks;
          cp_async16(sb + kk * kBPitch + 16 * c, B + static_cast<int64_t>(k + kk) * p.ldb + (ok ? 8 * c : 0), ok);
        }
      } else {
#pragma unroll
        for (int q = threadIdx.x; q < RP * 8; q += MS_THREADS) {
          const int j = q >> 3, c = q & 7;
          const bool ok = j < ranks;
          cp_async16(sb + j * kBPitch + 16 * c, B + static_cast<int64_t>(ok ? j : 0) * p.ldb + k + 8 * c, ok);
        }
      }
#pragma unroll
      for (int i = 0; i < 4; ++i)  // rows past the group's end are not read: their sums are not stored
        if (16 * i + mine < tile.rows)
          cp_async16(st + (16 * i + mine) * MS_PITCH + 16 * (threadIdx.x & 7), arow[i] + k, true);
    }
    cp_async_commit();
  };
  float acc[RP / 8][4], sum[RP / 8][4];
#pragma unroll
  for (int j = 0; j < RP / 8; ++j)
#pragma unroll
    for (int c = 0; c < 4; ++c) acc[j][c] = sum[j][c] = 0.0f;
#pragma unroll
  for (int s = 0; s < kStages - 1; ++s) load(s);
  const bool live = 16 * warp < tile.rows;
  for (int s = 0; s < steps; ++s) {
    cp_async_wait<kStages - 2>();
    __syncthreads();  // stage s has landed for all, and stage s - 1 has been read by all
    load(s + kStages - 1);
    if (!live) continue;
    const uint32_t sa = base + (s % kStages) * kStage;
    const uint32_t sb = sa + MP_TILE * MS_PITCH;
#pragma unroll
    for (int kk = 0; kk < MS_K; kk += 16) {
      uint32_t a[4];
      ldsm4(sa + (16 * warp + (lane & 15)) * MS_PITCH + (kk + 8 * (lane >> 4)) * 2, a);
#pragma unroll
      for (int j = 0; j < RP / 16; ++j) {
        uint32_t b[4];
        if constexpr (kKN)
          ldsm4_t(sb + (kk + (lane & 15)) * kBPitch + (16 * j + 8 * (lane >> 4)) * 2, b);
        else
          ldsm4(sb + (16 * j + (lane & 7) + 8 * (lane >> 4)) * kBPitch + (kk + 8 * ((lane >> 3) & 1)) * 2, b);
        mma_16816_bf16(acc[2 * j], a[0], a[1], a[2], a[3], b[0], b[1]);
        mma_16816_bf16(acc[2 * j + 1], a[0], a[1], a[2], a[3], b[2], b[3]);
      }
    }
    if ((s + 1) % MS_CHAIN == 0 || s + 1 == steps) {
#pragma unroll
      for (int j = 0; j < RP / 8; ++j)
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          sum[j][c] += acc[j][c];
          acc[j][c] = 0.0f;
        }
    }
  }
  cp_async_wait<0>();
  pdl_wait();  // what ran before may still read the parts of an earlier product
  if (!live) return;
  float* out = p.P + static_cast<int64_t>(blockIdx.y) * v.M * p.r + j0;
#pragma unroll
  for (int hh = 0; hh < 2; ++hh) {
    const int rr = 16 * warp + 8 * hh + (lane >> 2);
    if (rr >= tile.rows) continue;
    float* o = out + static_cast<int64_t>(tile.row0 + rr) * p.r + 2 * (lane & 3);
#pragma unroll
    for (int j = 0; j < RP / 8; ++j)
      if (8 * j < ranks) *reinterpret_cast<float2*>(o + 8 * j) = make_float2(sum[j][2 * hh], sum[j][2 * hh + 1]);
  }
}

// Fills the slots of T (or U): the sum of the K parts in order, or a T given by
// the caller, times the adapter's scale, as `parts` bf16 terms: two keep 16 bits
// of the value, 256 times finer than a bf16 result; three keep 24, for fp32
// results (those of the W' product, and the sums over tokens).  Also writes T itself in the
// batch's order, zero for tokens without adapter.  blockIdx.x < max_slots: 64
// rows (blockIdx.y) of a slot; above: the rows without adapter of a tile.
struct PackJob {
  const float* P;     // [splits][M][r], sorted rows, or null
  const float* given; // [M][r], batch order (P null)
  float* T;           // [M][r], batch order, or null
  uint16_t* slots;    // [slots][256][parts * rp]
  int splits;
};

struct PackParams {
  PackJob job[2];
  const float* s;   // [n]
  int r, rp, parts;
  int max_slots;
  unsigned* zero[2];  // arrival counters of the kernels that follow, set to 0
  int zero_len[2];
};

__global__ void __launch_bounds__(256) multi_pack_kernel(const PackParams p, const PlanView v) {
  const PackJob job = blockIdx.z == 0 ? p.job[0] : p.job[1];
  const int slot = blockIdx.x;
  pdl_launch_dependents();
  if (blockIdx.x == 0 && blockIdx.y == 0 && blockIdx.z == 0) {
    pdl_wait();
    for (int k = 0; k < 2; ++k)
      for (int i = threadIdx.x; i < p.zero_len[k]; i += blockDim.x) p.zero[k][i] = 0;
  }
  if (slot >= p.max_slots) {
    pdl_wait();
    if (!job.T) return;
    const int row0 = (slot - p.max_slots) * MP_SLOT_ROWS + 64 * blockIdx.y;
    const int vec = p.r / 4;
    for (int q = threadIdx.x; q < 64 * vec; q += blockDim.x) {
      const int i = row0 + q / vec;
      if (i < v.M && v.owner[i] < 0)
        reinterpret_cast<float4*>(job.T + static_cast<int64_t>(i) * p.r)[q % vec] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
    return;
  }
  const PlanSlot ps = plan_load(v.slots + slot);  // garbage past head->slots
  if (slot >= __ldg(&v.head->slots)) {
    pdl_wait();
    return;
  }
  const int g0 = ps.start, g1 = ps.end;
  const float s = __ldg(p.s + ps.adapter);
  const int row0 = ps.tile * MP_SLOT_ROWS;
  const int vec = p.rp / 4;
  pdl_wait();  // the parts of the product
  const int64_t part = static_cast<int64_t>(v.M) * p.r;
  for (int q = threadIdx.x; q < 64 * vec; q += blockDim.x) {
    const int rr = 64 * blockIdx.y + q / vec, c = 4 * (q % vec);
    const int at = row0 + rr;
    float x[4] = {0.f, 0.f, 0.f, 0.f};
    if (at >= g0 && at < g1 && c < p.r) {
      const int64_t orig = __ldg(v.perm + at);
      if (job.P) {
        const float* src = job.P + static_cast<int64_t>(at) * p.r + c;
#pragma unroll 4
        for (int k = 0; k < job.splits; ++k) {
          const float4 f = __ldcg(reinterpret_cast<const float4*>(src + k * part));
          x[0] += f.x, x[1] += f.y, x[2] += f.z, x[3] += f.w;
        }
      } else {
        const float4 f = *reinterpret_cast<const float4*>(job.given + orig * p.r + c);
        x[0] = f.x, x[1] = f.y, x[2] = f.z, x[3] = f.w;
      }
      if (job.T) *reinterpret_cast<float4*>(job.T + orig * p.r + c) = make_float4(x[0], x[1], x[2], x[3]);
#pragma unroll
      for (int j = 0; j < 4; ++j) x[j] *= s;
    }
    uint16_t* dst = job.slots + (static_cast<int64_t>(slot) * MP_SLOT_ROWS + rr) * (p.parts * p.rp) + c;
    for (int k = 0; k < p.parts; ++k) {
      const uint32_t lo = pack_bf16x2(x[0], x[1]), hi = pack_bf16x2(x[2], x[3]);
      *reinterpret_cast<uint2*>(dst + k * p.rp) = make_uint2(lo, hi);
      const float f[4] = {__uint_as_float(lo << 16), __uint_as_float(lo & 0xFFFF0000u), __uint_as_float(hi << 16),
                          __uint_as_float(hi & 0xFFFF0000u)};
      // an infinity or a NaN is its first part alone
#pragma unroll
      for (int j = 0; j < 4; ++j) x[j] = isfinite(f[j]) ? x[j] - f[j] : 0.0f;
    }
  }
}

// ====================================================================== adapters of a decode batch

// The adapter term of a batch of up to 32 tokens, added to the finished base
// product: Y[i] = acc[i] + s[a] sum_j T[i][j] L2[a][j] for one group
// (blockIdx.y) and a share of the columns (blockIdx.x); blockIdx.y = max_groups:
// the tokens without adapter.  L2 is the only large operand (2 r o bytes an
// adapter), read once for up to two tokens: the block's threads are S slices of
// the ranks by 256 / S column vectors of 8, eight rows a thread in flight, the
// first of them loaded before the wait for the base product; the slices are added
// through shared memory in order.  Few slices leave few blocks, each with more
// loads: 16 adapters of rank 64 and 22016 columns take 20 us with 16 slices (2752
// blocks, whose set-up is most of it) and 12 with 4; a single token of 4096
// columns needs the 16 to have 32 blocks at all.
// A kernel of its own and not a share of the decode kernel's warps: three warps an
// SM cannot keep enough loads in flight beside a ring that fills the shared memory
// (the same 16 adapters: 114 to 140 us for the two in one kernel, 59 for the
// weight stream alone).
constexpr int MX_THREADS = 256;
constexpr int MX_MT = 2;
constexpr int MX_ROWS = 8;
constexpr int mx_cols(int slices) { return MX_THREADS / slices * 8; }

struct ExpandParams {
  const float* P;      // [parts][M][r] of T, sorted rows
  const uint16_t* L2;  // bank [n][r][N]
  const float* s;      // [n]
  const float* acc;    // [M][N] base product
  void* Y;             // [M][N], fp32 (may be acc) or bf16
  float* T;            // [M][r], batch order, or null
  int parts, r, N, max_groups;
};

template <bool kBf16, int S>
__global__ void __launch_bounds__(MX_THREADS, 3) multi_expand_kernel(const ExpandParams p, const PlanView v) {
  constexpr int kVecs = MX_THREADS / S, kCols = mx_cols(S);
  __shared__ __align__(16) float Ts[MX_MT * QLORA_MAX_RANK];
  __shared__ __align__(16) float red[MX_MT * MX_THREADS * 8];  // [token][slice][column]
  const int tid = threadIdx.x;
  const int64_t n0 = static_cast<int64_t>(blockIdx.x) * kCols;
  const int cols = static_cast<int>(p.N - n0 < kCols ? p.N - n0 : kCols);  // a multiple of 64
  if (static_cast<int>(blockIdx.y) == p.max_groups) {
    pdl_wait();
    for (int m = 0; m < v.M; ++m) {
      if (v.owner[m] >= 0) continue;
      if (p.T && blockIdx.x == 0)
        for (int j = tid; j < p.r; j += MX_THREADS) p.T[static_cast<int64_t>(m) * p.r + j] = 0.0f;
      if constexpr (kBf16)
        for (int c = tid; c < cols; c += MX_THREADS) {
          const int64_t at = static_cast<int64_t>(m) * p.N + n0 + c;
          static_cast<uint16_t*>(p.Y)[at] = __bfloat16_as_ushort(__float2bfloat16_rn(p.acc[at]));
        }
    }
    return;
  }
  const PlanGroup pg = plan_load(v.groups + blockIdx.y);  // garbage past head->groups
  if (static_cast<int>(blockIdx.y) >= __ldg(&v.head->groups)) {
    pdl_wait();
    return;
  }
  const int a = pg.adapter, g0 = pg.start, g1 = pg.end;
  const float s = __ldg(p.s + a);
  const int vec = tid % kVecs, slice = tid / kVecs;
  const bool in = 8 * vec < cols;
  const uint16_t* L2 = p.L2 + static_cast<int64_t>(a) * p.r * p.N + n0 + 8 * vec;
  auto load = [&](int j0, uint4 (&w)[MX_ROWS]) {
#pragma unroll
    for (int u = 0; u < MX_ROWS; ++u) {
      const int j = j0 + slice + u * S;
      w[u] = in && j < p.r ? __ldg(reinterpret_cast<const uint4*>(L2 + static_cast<int64_t>(j) * p.N))
                           : make_uint4(0u, 0u, 0u, 0u);
    }
  };
  uint4 w[MX_ROWS];
  load(0, w);
  pdl_wait();
  for (int m0 = g0; m0 < g1; m0 += MX_MT) {
    const int mt = min(MX_MT, g1 - m0);
    // T of these tokens: groups of threads take every sub-th part, then the groups are added in order
    const int nt4 = mt * p.r / 4;  // float4s, 2 .. 256
    const int subs = min(MX_THREADS / nt4, p.parts);
    const int q = tid % nt4, sub = tid / nt4;
    if (sub < subs) {
      const float4* src = reinterpret_cast<const float4*>(p.P + static_cast<int64_t>(m0) * p.r) + q;
      const int64_t part4 = static_cast<int64_t>(v.M) * p.r / 4;
      float4 f = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
      for (int k = sub; k < p.parts; k += subs) {
        const float4 x = __ldcg(src + k * part4);
        f.x += x.x, f.y += x.y, f.z += x.z, f.w += x.w;
      }
      reinterpret_cast<float4*>(red)[sub * nt4 + q] = f;
    }
    __syncthreads();
    if (tid < nt4) {
      float4 f = make_float4(0.f, 0.f, 0.f, 0.f);
      for (int k = 0; k < subs; ++k) {
        const float4 x = reinterpret_cast<const float4*>(red)[k * nt4 + tid];
        f.x += x.x, f.y += x.y, f.z += x.z, f.w += x.w;
      }
      reinterpret_cast<float4*>(Ts)[tid] = f;
      if (p.T && blockIdx.x == 0)
        reinterpret_cast<float4*>(p.T + static_cast<int64_t>(v.perm[m0 + 4 * tid / p.r]) * p.r)[tid % (p.r / 4)] = f;
    }
    __syncthreads();
    float acc[MX_MT][8];
#pragma unroll
    for (int m = 0; m < MX_MT; ++m)
#pragma unroll
      for (int c = 0; c < 8; ++c) acc[m][c] = 0.0f;
    for (int j0 = 0; j0 < p.r; j0 += MX_ROWS * S) {
      if (j0 > 0 || m0 > g0) load(j0, w);
#pragma unroll
      for (int u = 0; u < MX_ROWS; ++u) {
        const int j = j0 + slice + u * S;
        if (j >= p.r) break;
        const uint32_t ws[4] = {w[u].x, w[u].y, w[u].z, w[u].w};
#pragma unroll
        for (int m = 0; m < MX_MT; ++m) {
          if (m >= mt) break;
          const float t = Ts[m * p.r + j];
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            acc[m][2 * c] = fmaf(t, __uint_as_float(ws[c] << 16), acc[m][2 * c]);
            acc[m][2 * c + 1] = fmaf(t, __uint_as_float(ws[c] & 0xFFFF0000u), acc[m][2 * c + 1]);
          }
        }
      }
    }
#pragma unroll
    for (int m = 0; m < MX_MT; ++m) {
      if (m >= mt) break;
      float4* d = reinterpret_cast<float4*>(red + (m * S + slice) * kCols + 8 * vec);
      d[0] = make_float4(acc[m][0], acc[m][1], acc[m][2], acc[m][3]);
      d[1] = make_float4(acc[m][4], acc[m][5], acc[m][6], acc[m][7]);
    }
    __syncthreads();
    for (int e = tid; e < mt * (kCols / 4); e += MX_THREADS) {  // four columns of a token a thread
      const int m = e / (kCols / 4), c = 4 * (e % (kCols / 4));
      if (c >= cols) continue;
      const int64_t at = static_cast<int64_t>(v.perm[m0 + m]) * p.N + n0 + c;
      const float4 base = *reinterpret_cast<const float4*>(p.acc + at);
      float4 f = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int k = 0; k < S; ++k) {
        const float4 x = *reinterpret_cast<const float4*>(red + (m * S + k) * kCols + c);
        f.x += x.x, f.y += x.y, f.z += x.z, f.w += x.w;
      }
      f = make_float4(fmaf(s, f.x, base.x), fmaf(s, f.y, base.y), fmaf(s, f.z, base.z), fmaf(s, f.w, base.w));
      if constexpr (kBf16)
        *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.Y) + at) =
            make_uint2(pack_bf16x2(f.x, f.y), pack_bf16x2(f.z, f.w));
      else
        *reinterpret_cast<float4*>(static_cast<float*>(p.Y) + at) = f;
    }
    __syncthreads();
  }
}

// ====================================================================== W' product with the groups' terms

__device__ __forceinline__ void tma_load_3d_pair(void* smem_dst, const CUtensorMap* map, uint32_t bar, int32_t x,
                                                 int32_t y, int32_t z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(smem_u32(smem_dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y), "r"(z)
      : "memory");
}

struct MultiPairParams {
  PairGemmParams g;         // k_ext_stages is not used: a tile has slot_stages stages per slot
  int even;                 // no whole rounds: the stages of all tiles in even shares (see below)
  int chain;                // stages of an accumulator
  int slot_stages;          // two (part, 64 ranks) pairs each
  int rp, parts;            // of the slots
  int used;                 // the parts that enter the product, 2 or 3
  const uint16_t* A;        // [M][K], batch order
  const uint16_t* Wd;       // W'^T [o][h]
  const uint16_t* slots;
  const uint16_t* bank;     // forward: L2 [n][r][o]; backward: L1 [n][h][r]
  int K, r;
};

__device__ __forceinline__ float dot8(uint4 a, uint4 b, float x) {
  const uint32_t aw[4] = {a.x, a.y, a.z, a.w}, bw[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x = fmaf(__uint_as_float(aw[i] << 16), __uint_as_float(bw[i] << 16), x);
    x = fmaf(__uint_as_float(aw[i] & 0xFFFF0000u), __uint_as_float(bw[i] & 0xFFFF0000u), x);
  }
  return x;
}

// x += a w for eight columns.
__device__ __forceinline__ void axpy8(float a, uint4 w, float (&x)[8]) {
  const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    x[2 * c] = fmaf(a, __uint_as_float(ws[c] << 16), x[2 * c]);
    x[2 * c + 1] = fmaf(a, __uint_as_float(ws[c] & 0xFFFF0000u), x[2 * c + 1]);
  }
}

// The slot row of sorted row m, or null for a row without adapter, and its adapter.
__device__ __forceinline__ const uint16_t* slot_row(const MultiPairParams& p, const PlanView& v, int m, int& adapter) {
  const int t = m / MP_SLOT_ROWS;
  for (int s = v.tile_slot0[t]; s < v.tile_slot0[t + 1]; ++s) {
    const PlanSlot ps = plan_load(v.slots + s);
    if (m < ps.start || m >= ps.end) continue;
    adapter = ps.adapter;
    return p.slots + (static_cast<int64_t>(s) * MP_SLOT_ROWS + m % MP_SLOT_ROWS) * (p.parts * p.rp);
  }
  return nullptr;
}

// Eight elements n .. n + 7 from their own row and adapter alone, in fp32: the base sum,
template <bool kBwd>
__device__ __forceinline__ void base_elements(const MultiPairParams& p, const uint16_t* a, int n, float (&x)[8]) {
#pragma unroll
  for (int c = 0; c < 8; ++c) x[c] = 0.0f;
  for (int k = 0; k < p.K; k += 8) {  // K is a multiple of 64
    const uint4 av = *reinterpret_cast<const uint4*>(a + k);
    if (kBwd) {
      const uint32_t as[4] = {av.x, av.y, av.z, av.w};
#pragma unroll
      for (int i = 0; i < 8; ++i)
        axpy8(__uint_as_float(i & 1 ? as[i / 2] & 0xFFFF0000u : as[i / 2] << 16),
              *reinterpret_cast<const uint4*>(p.Wd + static_cast<int64_t>(k + i) * p.g.N + n), x);
    } else {
#pragma unroll
      for (int c = 0; c < 8; ++c)
        x[c] = dot8(av, *reinterpret_cast<const uint4*>(p.Wd + static_cast<int64_t>(n + c) * p.K + k), x[c]);
    }
  }
}

// and the adapter's term.
template <bool kBwd>
__device__ __forceinline__ void adapter_elements(const MultiPairParams& p, const uint16_t* row, int adapter, int n,
                                                 float (&d)[8]) {
  const uint16_t* b = p.bank + static_cast<int64_t>(adapter) * p.r * p.g.N;
#pragma unroll
  for (int c = 0; c < 8; ++c) d[c] = 0.0f;
  for (int j = 0; j < p.r; ++j) {
    float t = bf16_bits_to_float(row[j]) + bf16_bits_to_float(row[p.rp + j]);
    if (p.used > 2) t += bf16_bits_to_float(row[2 * p.rp + j]);
    if (kBwd) {
#pragma unroll
      for (int c = 0; c < 8; ++c) d[c] = fmaf(t, bf16_bits_to_float(b[static_cast<int64_t>(n + c) * p.r + j]), d[c]);
    } else {
      axpy8(t, *reinterpret_cast<const uint4*>(b + static_cast<int64_t>(j) * p.g.N + n), d);
    }
  }
}

// Whether all of x is finite: x 0 is 0 then, so one fused multiply-add each tells.
template <int kN>
__device__ __forceinline__ bool all_finite(const float* x) {
  float z = 0.0f;
#pragma unroll
  for (int t = 0; t < kN; ++t) z = fmaf(x[t], 0.0f, z);
  return z == 0.0f;
}

// Replaces what is not finite among the `len` elements (a multiple of 8) from n on that this thread
// has stored of sorted row m by its own sum.  Nothing to do in a tile without adapters, nor where the
// row, or its product with its adapter's first factor, holds a NaN: all its elements are NaN then,
// whatever W' and the factors are.  Where the adapter's term is NaN, so is the element, without the long
// sum.  So a batch of NaN costs a look at its rows (4096 x 4096 x 11008: nothing to be seen) and one with
// an infinity in every row 5 ms; neighbours of one adapter of infinities take the long sum, eight
// elements at a time, so that each load of the row and of W' serves eight: 8 ms, the backward 12.  Never
// inlined: the path is rare and long.
template <bool kBwd>
__device__ __noinline__ void multi_repair(const MultiPairParams& p, const PlanView& v, int m, int n, int len) {
  const uint16_t* a = p.A + static_cast<int64_t>(v.perm[m]) * p.K;
  const int tile = m / MP_SLOT_ROWS;
  if (v.tile_slot0[tile] == v.tile_slot0[tile + 1]) return;
  int adapter = -1;
  const uint16_t* row = slot_row(p, v, m, adapter);
  if (row)
    for (int j = 0; j < p.r; ++j)
      if (isnan(bf16_bits_to_float(row[j]))) return;
  for (int k = 0; k < p.K; k += 8) {
    const uint4 x = *reinterpret_cast<const uint4*>(a + k);
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (isnan(__uint_as_float(w[i] << 16)) || isnan(__uint_as_float(w[i] & 0xFFFF0000u))) return;
  }
  const int64_t at = static_cast<int64_t>(v.perm[m]) * p.g.ld_out + n;
  uint16_t* o16 = static_cast<uint16_t*>(p.g.out) + at;
  float* o32 = static_cast<float*>(p.g.out) + at;
  for (int t = 0; t < len; t += 8) {
    unsigned bad = 0;
    for (int c = 0; c < 8; ++c)
      if (!isfinite(p.g.out_bf16 ? bf16_bits_to_float(o16[t + c]) : o32[t + c])) bad |= 1u << c;
    if (bad == 0) continue;
    float x[8], d[8] = {};
    if (row) adapter_elements<kBwd>(p, row, adapter, n + t, d);
    bool any = false;
#pragma unroll
    for (int c = 0; c < 8; ++c) any = any || ((bad >> c & 1) && !isnan(d[c]));
    if (any) {
      base_elements<kBwd>(p, a, n + t, x);
#pragma unroll
      for (int c = 0; c < 8; ++c) d[c] += x[c];
    }
#pragma unroll
    for (int c = 0; c < 8; ++c) {
      if (!(bad >> c & 1)) continue;
      if (p.g.out_bf16)
        o16[t + c] = __bfloat16_as_ushort(__float2bfloat16_rn(d[c]));
      else
        o32[t + c] = d[c];
    }
  }
}

// Fewer tiles than SM pairs (`even`): the K stages of all tiles, one tile after
// the other, are dealt out in equal contiguous shares, so that every pair works
// for the same time whatever the number of tiles and of slots in them (333
// tokens, 13824 x 5120, 40 tiles on 74 pairs: the call takes 165 us with one tile
// a pair, 130 so).  A share's first and last tile may be partial: their sums go to
// the pair's two places of the partial buffer, and multi_reduce_kernel adds the
// places of a tile in order.
struct StageShare {
  int64_t lo, hi;  // stages of this pair
};
__device__ __forceinline__ StageShare stage_share(int64_t total, int pair, int pairs) {
  return {total * pair / pairs, total * (pair + 1) / pairs};
}

struct PairTiles {
  int m_tiles, n_tiles;
  __device__ __forceinline__ void at(int u, int& mt, int& n0) const {
    const int band = u / (PG_BAND * m_tiles);
    const int r = u - band * PG_BAND * m_tiles;
    const int width = min(PG_BAND, n_tiles - band * PG_BAND);
    mt = r / width;
    n0 = (band * PG_BAND + r % width) * PG_BN;
  }
};

// Stages of tile u.
__device__ __forceinline__ int tile_stages(const MultiPairParams& p, const PlanView& v, int u) {
  const PairTiles tiles{p.g.units / p.g.n_tiles, p.g.n_tiles};
  int mt, n0;
  tiles.at(u, mt, n0);
  return p.g.k_main_stages + (v.tile_slot0[mt + 1] - v.tile_slot0[mt]) * p.slot_stages;
}

// Calls f(u, first stage, stages) for all tiles, by one warp; returns the sum of the stages.
template <typename F>
__device__ __forceinline__ int64_t walk_tiles(const MultiPairParams& p, const PlanView& v, F f) {
  const int lane = threadIdx.x & 31;
  int64_t carry = 0;
  for (int b = 0; b < p.g.units; b += 32) {
    const int u = b + lane;
    const int n = u < p.g.units ? tile_stages(p, v, u) : 0;
    int s = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(0xFFFFFFFFu, s, o);
      if (lane >= o) s += x;
    }
    f(u, carry + s - n, n);
    carry += __shfl_sync(0xFFFFFFFFu, s, 31);
  }
  return carry;
}

// A piece of a tile that a pair computes.
struct PairItem {
  int mt, n0, kbeg, kend;
  int slot0;  // first slot of the tile
  int part;   // place in the partial buffer (-1: the whole tile)
};
constexpr int MG_PAIR_ITEMS = 128;  // pieces of an even share: at most the tiles, which are fewer than the pairs
constexpr int MG_PAIR_SMEM = PG_SMEM_BYTES + 16 + MG_PAIR_ITEMS * static_cast<int>(sizeof(PairItem));

// pair_gemm_kernel's pipeline (256 x 256 tiles on two-SM clusters, 128-deep
// stages, two accumulators, K parts for what does not fill a round) with K
// extended per tile, by slot_stages stages for every slot of the tile.  The halves of a
// stage are 64 ranks of one bf16 part of the slot (A) and the same 64 ranks of the group's
// factor (B), straight from the bank (the forward's L2 is an N-major operand, the
// backward's L1 a K-major one; ranks past r are zero-filled by the 3-D map): [hi | mid] of
// 64 ranks for a bf16 result, hi, mid and lo one after the other for an fp32 one, whose
// last stage may be half zeros.
// Rows are read in sorted order and written to their own place.
// The tensor core cuts its running sum to fp32 at every step (16 products), which
// adds up over a long accumulator: 11e-6 against 64 bits at K = 11008, where an
// fp32 sum is 1e-6 off, and a bf16 result then rounds to another value in 0.6 % of
// the elements of a sum of 8192 positive products.  So the accumulator changes every
// `chain` stages of 128 products, and the epilogue, eight warps with 128 sums a
// thread, adds it in registers while the MMAs go on with the other one.  (Running
// sums in memory instead, 256 KB a pair in L2: 453 us for 345 at 4096 x 4096 x 11008.)
//   bf16 results: 8 stages (0.07 % there).  One accumulator: 289 us a cold call of 4096 x
//   4096 x 11008, 16 stages 293, 8 stages 301, 4 stages 328.
//   fp32 results: as exact as an fp32 sum.  4 stages, 3.4e-7 (fp32 sums of K = 4096:
//   5.1e-7), 368 us cold for 344 with 8 stages (7.4e-7); up to K = 2048, where an fp32 sum
//   is better than that (1.6e-7 at 768) and the product a smaller part of the call, 2
//   stages, 1.9e-7 (4096 x 4096 x 11008 would take 405 us).
constexpr int multi_chain(bool out_bf16, int64_t K) { return out_bf16 ? 8 : (K > 2048 ? 4 : 2); }
constexpr int MG_EPI_WARPS = 8;
constexpr int MG_PAIR_THREADS = 64 + 32 * MG_EPI_WARPS;
constexpr int MG_COLS = PG_ACC_COLS / 2;  // columns of an epilogue warp
template <bool kBwd>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(MG_PAIR_THREADS, 1)
    multi_pair_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmAs,
                      const __grid_constant__ CUtensorMap tmB, const __grid_constant__ CUtensorMap tmAe,
                      const __grid_constant__ CUtensorMap tmBe, const __grid_constant__ MultiPairParams mp,
                      const __grid_constant__ PlanView v) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sA = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint8_t* sB = sA + PG_STAGES * PG_OPND_BYTES;
  uint64_t* bars = reinterpret_cast<uint64_t*>(sB + PG_STAGES * PG_OPND_BYTES);
  uint64_t* full = bars;                 // even CTA: TMA bytes of both CTAs (+ its producer)
  uint64_t* empty = full + PG_STAGES;    // each CTA: the MMA's commit
  uint64_t* tfull = empty + PG_STAGES;   // each CTA: accumulator complete
  uint64_t* tempty = tfull + 2;          // even CTA: the epilogue warps of the pair
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(tempty + 2);
  int* n_even = reinterpret_cast<int*>(reinterpret_cast<uint8_t*>(bars) + PG_BAR_BYTES);
  PairItem* even = reinterpret_cast<PairItem*>(n_even + 4);

  const PairGemmParams& p = mp.g;
  const uint32_t rank = cluster_ctarank();
  const int pair = static_cast<int>(cluster_index_x());
  const int npairs = static_cast<int>(cluster_count_x());
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int KM = p.k_main_stages;
  const PairTiles tiles{p.units / p.n_tiles, p.n_tiles};
  const int n_parts = (p.units - p.full_units) * p.split;
  const int n_items = p.full_units + n_parts;
  auto item_of = [&](int k) -> PairItem {
    if (mp.even) return even[k];
    const int u = pair + k * npairs;
    PairItem it;
    it.part = u >= n_parts ? -1 : u;
    tiles.at(u >= n_parts ? u - n_parts : p.full_units + u / p.split, it.mt, it.n0);
    it.slot0 = v.tile_slot0[it.mt];
    const int S = KM + (v.tile_slot0[it.mt + 1] - it.slot0) * mp.slot_stages;
    it.kbeg = 0;
    it.kend = S;
    if (it.part >= 0) {
      const int64_t j = u % p.split;
      it.kbeg = static_cast<int>(j * S / p.split);
      it.kend = static_cast<int>((j + 1) * S / p.split);
    }
    return it;
  };
  if (mp.even && warp == 2) {
    const int64_t total = walk_tiles(mp, v, [](int, int64_t, int) {});
    const StageShare share = stage_share(total, pair, npairs);
    int count = 0;
    walk_tiles(mp, v, [&](int u, int64_t at, int n) {
      const bool mine = n > 0 && at < share.hi && at + n > share.lo;
      const unsigned who = __ballot_sync(0xFFFFFFFFu, mine);
      if (mine) {
        const int k = count + __popc(who & ((1u << lane) - 1u));
        PairItem it;
        tiles.at(u, it.mt, it.n0);
        it.kbeg = static_cast<int>(max(share.lo - at, static_cast<int64_t>(0)));
        it.kend = static_cast<int>(min(share.hi - at, static_cast<int64_t>(n)));
        it.slot0 = v.tile_slot0[it.mt];
        it.part = it.kbeg == 0 && it.kend == n ? -1 : 2 * pair + (at > share.lo ? 1 : 0);
        even[k] = it;
      }
      count += __popc(who);
    });
    if (lane == 0) *n_even = count;
  }

  if (threadIdx.x == 0) {
    for (int s = 0; s < PG_STAGES; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&tfull[b], 1);
      mbar_init(&tempty[b], 2 * MG_EPI_WARPS);
    }
    fence_mbar_init();
    tma_prefetch_map(&tmB);
    tma_prefetch_map(&tmAe);
    tma_prefetch_map(&tmBe);
  }
  if (warp == 1) {
    tmem_alloc_pair(tmem_slot, 2 * PG_ACC_COLS);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  cluster_barrier();  // both CTAs' barriers initialised and TMEM allocated
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  pdl_launch_dependents();
  pdl_wait();  // the slots, W' and the sorted rows
  const int nk = mp.even ? *n_even : (pair < n_items ? (n_items - 1 - pair) / npairs + 1 : 0);  // items of this pair

  if (warp == 0) {
    if (lane == 0) {
      // ---------------- TMA producer: this CTA's 128 rows of A and of B of a stage
      const CUtensorMap* ma = v.head->in_order ? &tmA : &tmAs;
      int G = 0;
      bool ok = true;
      for (int k = 0; k < nk && ok; ++k) {
        const PairItem it = item_of(k);
        const int m0 = it.mt * PG_BM + static_cast<int>(rank) * 128;
        const int n0 = it.n0 + static_cast<int>(rank) * 128;
        for (int i = it.kbeg; i < it.kend; ++i, ++G) {
          const int s = G % PG_STAGES;
          if (!mbar_wait_idle(&empty[s], ((G / PG_STAGES) & 1) ^ 1, kTagPgEmpty)) {
            ok = false;
            break;
          }
          const uint32_t fb = cluster_addr(&full[s], 0);
          uint8_t* a_dst = sA + s * PG_OPND_BYTES;
          uint8_t* b_dst = sB + s * PG_OPND_BYTES;
          if (rank == 0) mbar_arrive_expect_tx(&full[s], 4 * PG_OPND_BYTES);
          if (i < KM) {
            const int k0 = i * PG_BK;
            tma_load_2d_pair(a_dst, ma, fb, k0, m0);
            tma_load_2d_pair(a_dst + PG_ATOM_BYTES, ma, fb, k0 + 64, m0);
            if (kBwd) {
              tma_load_2d_pair(b_dst, &tmB, fb, n0, k0);
              tma_load_2d_pair(b_dst + PG_ATOM_BYTES, &tmB, fb, n0 + 64, k0);
            } else {
              tma_load_2d_pair(b_dst, &tmB, fb, k0, n0);
              tma_load_2d_pair(b_dst + PG_ATOM_BYTES, &tmB, fb, k0 + 64, n0);
            }
          } else {
            const int e = (i - KM) / mp.slot_stages;
            const int j0 = 2 * ((i - KM) - e * mp.slot_stages);
            const int slot = it.slot0 + e;
            const int a = __ldg(&v.slots[slot].adapter);
            const int y = slot * MP_SLOT_ROWS + static_cast<int>(rank) * 128;
            for (int h = 0; h < 2; ++h) {
              const int j = j0 + h, chunk = j / mp.used;
              // behind the last pair: past the end of both maps, which read zeros there
              const bool in = 64 * chunk < mp.rp;
              const int x = in ? 64 * chunk : mp.rp;
              tma_load_2d_pair(a_dst + h * PG_ATOM_BYTES, &tmAe, fb, in ? (j - chunk * mp.used) * mp.rp + x : mp.parts * mp.rp, y);
              if (kBwd) {
                // K-major: 64 ranks of 128 rows of L1
                tma_load_3d_pair(b_dst + h * PG_ATOM_BYTES, &tmBe, fb, x, n0, a);
              } else {
                // N-major: 64 ranks of each 64 columns of L2, the second half of the stage below the first
                for (int c = 0; c < 2; ++c)
                  tma_load_3d_pair(b_dst + c * PG_ATOM_BYTES + h * (PG_ATOM_BYTES / 2), &tmBe, fb, n0 + 64 * c, x, a);
              }
            }
          }
        }
      }
      // Leave no copy in flight: the even CTA's last phases count both CTAs' bytes.
      if (rank == 0)
        for (int g = G - PG_STAGES > 0 ? G - PG_STAGES : 0; g < G; ++g)
          mbar_wait_idle(&full[g % PG_STAGES], (g / PG_STAGES) & 1, kTagPgFull);
    }
  } else if (warp == 1) {
    if (rank == 0 && lane == 0) {
      // ---------------- MMA issuer (even CTA)
      uint64_t a_desc0[PG_STAGES], b_desc0[PG_STAGES], bmn_desc0[PG_STAGES];
#pragma unroll
      for (int s = 0; s < PG_STAGES; ++s) {
        a_desc0[s] = sw128_desc(smem_u32(sA + s * PG_OPND_BYTES), 16, 1024);
        b_desc0[s] = sw128_desc(smem_u32(sB + s * PG_OPND_BYTES), 16, 1024);
        bmn_desc0[s] = sw128_desc(smem_u32(sB + s * PG_OPND_BYTES), PG_ATOM_BYTES, 1024);
      }
      int G = 0, A = 0;  // stages and accumulators so far
      bool ok = true;
      for (int k = 0; k < nk && ok; ++k) {
        const PairItem it = item_of(k);
        for (int i = it.kbeg; i < it.kend && ok; ++A) {
          const int b = A & 1;
          if (!mbar_wait_idle<true>(&tempty[b], ((A >> 1) & 1) ^ 1, kTagPgTEmpty)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t d_tmem = tmem + static_cast<uint32_t>(b * PG_ACC_COLS);
          const int first = i, end = min(it.kend, i + mp.chain);
          for (; i < end; ++i, ++G) {
            const int s = G % PG_STAGES;
            if (!mbar_wait(&full[s], (G / PG_STAGES) & 1, kTagPgFull)) {
              ok = false;
              break;
            }
            tc_fence_after();
            const bool b_mn = kBwd == (i < KM);
            const uint64_t ad = s == 0 ? a_desc0[0] : (s == 1 ? a_desc0[1] : a_desc0[2]);
            const uint64_t bd = b_mn ? (s == 0 ? bmn_desc0[0] : (s == 1 ? bmn_desc0[1] : bmn_desc0[2]))
                                     : (s == 0 ? b_desc0[0] : (s == 1 ? b_desc0[1] : b_desc0[2]));
            const uint32_t idesc = idesc_bf16(PG_BM, PG_BN, false, false) | (b_mn ? 1u << 16 : 0u);
#pragma unroll
            for (int kk = 0; kk < PG_BK / 16; ++kk) {
              const uint32_t k_off = ((kk >> 2) * PG_ATOM_BYTES + (kk & 3) * 32) >> 4;
              const uint64_t adesc = ad + k_off;
              const uint64_t bdesc = bd + (b_mn ? static_cast<uint32_t>(kk * 2048 >> 4) : k_off);
              umma_bf16_pair(d_tmem, adesc, bdesc, idesc, (i > first || kk > 0) ? 1u : 0u);
            }
            umma_commit_pair(&empty[s], 0x3);
          }
          if (ok) umma_commit_pair(&tfull[b], 0x3);
        }
      }
    }
  } else {
    // ---------------- epilogue: thread = row (TMEM lane) of this CTA, warps 2 .. 5 the first 128
    // columns, warps 6 .. 9 the others; the sums of an item stay in registers
    const int q = warp & 3;
    const int c0 = (warp - 2) / 4 * MG_COLS;
    const int row = static_cast<int>(rank) * 128 + q * 32 + lane;  // row within the pair tile
    const uint32_t t_addr = tmem + (static_cast<uint32_t>(q * 32) << 16) + static_cast<uint32_t>(c0);
    int A = 0;
    bool ok = true;
    for (int k = 0; k < nk && ok; ++k) {
      const PairItem it = item_of(k);
      const int m = it.mt * PG_BM + row;
      const int64_t to = m < p.M ? v.perm[m] : 0;
      float x[MG_COLS];
#pragma unroll
      for (int j = 0; j < MG_COLS; ++j) x[j] = 0.0f;
      for (int i = it.kbeg; i < it.kend; ++A) {
        const int b = A & 1;
        if (!__all_sync(0xFFFFFFFFu, mbar_wait_idle(&tfull[b], (A >> 1) & 1, kTagPgTFull))) {
          ok = false;
          break;
        }
        tc_fence_after();
#pragma unroll
        for (int c = 0; c < MG_COLS; c += 16) {
          uint32_t r[16];
          tmem_ld16(t_addr + static_cast<uint32_t>(b * PG_ACC_COLS + c), r);
          tmem_ld_wait();
#pragma unroll
          for (int t = 0; t < 16; ++t) x[c + t] += __uint_as_float(r[t]);
        }
        // the accumulator is in registers: hand it back to the MMA issuer
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_even(&tempty[b], rank);
        i = min(it.kend, i + mp.chain);
      }
      if (!ok) break;
      const int n0 = it.n0 + c0;
      if (it.part >= 0) {
        // [4 columns][row]: a warp's 32 rows are 512 contiguous bytes
        float4* dst = reinterpret_cast<float4*>(p.partial + static_cast<int64_t>(it.part) * PG_BM * PG_BN) +
                      c0 / 4 * PG_BM + row;
        if (m < p.M)
#pragma unroll
          for (int j = 0; j < MG_COLS; j += 4) dst[j / 4 * PG_BM] = make_float4(x[j], x[j + 1], x[j + 2], x[j + 3]);
        if (mp.even) continue;
        // the warp that completes the last part of a tile adds the parts in order
        __threadfence();
        __syncwarp();
        const int tail = it.part / p.split;
        unsigned prior = 0;
        if (lane == 0)
          prior = atomicAdd(&p.counters[(tail * 2 + static_cast<int>(rank)) * MG_EPI_WARPS + warp - 2], 1u);
        prior = __shfl_sync(0xFFFFFFFFu, prior, 0);
        if (prior != static_cast<unsigned>(p.split - 1)) continue;
        __threadfence();
        const float4* src =
            reinterpret_cast<const float4*>(p.partial + static_cast<int64_t>(tail) * p.split * PG_BM * PG_BN) +
            c0 / 4 * PG_BM + row;
#pragma unroll
        for (int j = 0; j < MG_COLS; ++j) x[j] = 0.0f;
        if (m < p.M)
          for (int s = 0; s < p.split; ++s)
#pragma unroll
            for (int j = 0; j < MG_COLS; j += 4) {
              const float4 a = __ldcg(src + static_cast<int64_t>(s) * (PG_BM * PG_BN / 4) + j / 4 * PG_BM);
              x[j] += a.x, x[j + 1] += a.y, x[j + 2] += a.z, x[j + 3] += a.w;
            }
      }
      if (m >= p.M) continue;
      if (p.out_bf16) {
        uint16_t* out = static_cast<uint16_t*>(p.out) + to * p.ld_out + n0;
#pragma unroll
        for (int j = 0; j < MG_COLS; j += 8)
          if (n0 + j < p.N)
            __stcs(reinterpret_cast<uint4*>(out + j),
                   make_uint4(pack_bf16x2(x[j], x[j + 1]), pack_bf16x2(x[j + 2], x[j + 3]),
                              pack_bf16x2(x[j + 4], x[j + 5]), pack_bf16x2(x[j + 6], x[j + 7])));
      } else {
        float* out = static_cast<float*>(p.out) + to * p.ld_out + n0;
#pragma unroll
        for (int j = 0; j < MG_COLS; j += 4)
          if (n0 + j < p.N) __stcs(reinterpret_cast<float4*>(out + j), make_float4(x[j], x[j + 1], x[j + 2], x[j + 3]));
      }
      if (!all_finite<MG_COLS>(x)) multi_repair<kBwd>(mp, v, m, n0, min(MG_COLS, p.N - n0));
    }
  }

  __syncwarp();
  tc_fence_before();
  cluster_barrier();  // no CTA leaves while the other may still touch its barriers or TMEM
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, 2 * PG_ACC_COLS);
  }
}

// Adds the partial sums of the tiles that several pairs computed, in the order
// of their stages.  blockIdx.x: tile, blockIdx.y: 16 of its rows.
constexpr int MR_ROWS = 16;
template <bool kBwd>
__global__ void __launch_bounds__(256) multi_reduce_kernel(const __grid_constant__ MultiPairParams mp, int pairs,
                                                           const __grid_constant__ PlanView v) {
  __shared__ int64_t at, all;
  __shared__ int len;
  const PairGemmParams& p = mp.g;
  const int u = blockIdx.x;
  int mt, n0;
  PairTiles{p.units / p.n_tiles, p.n_tiles}.at(u, mt, n0);
  const int m0 = mt * PG_BM + MR_ROWS * static_cast<int>(blockIdx.y);
  pdl_launch_dependents();
  if (m0 >= p.M) {
    pdl_wait();
    return;
  }
  if (threadIdx.x < 32) {
    const int64_t total = walk_tiles(mp, v, [&](int t, int64_t first, int n) {
      if (t == u) at = first, len = n;
    });
    if (threadIdx.x == 0) all = total;
  }
  __syncthreads();
  // the first and last pair with stages of this tile, and the place of the first's sum
  int c0 = static_cast<int>(at * pairs / all);
  while (stage_share(all, c0, pairs).hi <= at) ++c0;
  while (c0 > 0 && stage_share(all, c0, pairs).lo > at) --c0;
  int c1 = c0;
  while (stage_share(all, c1, pairs).hi < at + len) ++c1;
  pdl_wait();
  if (c0 == c1) return;  // one pair computed the whole tile and has stored it
  const int64_t place0 = 2 * c0 + (at > stage_share(all, c0, pairs).lo ? 1 : 0);
  const float4* first = reinterpret_cast<const float4*>(p.partial + place0 * PG_BM * PG_BN);
  const float4* rest = reinterpret_cast<const float4*>(p.partial);
  // 8 columns of a row a thread; the places are [4 columns][row]
  for (int q = threadIdx.x; q < MR_ROWS * PG_BN / 8; q += 256) {
    const int m = m0 + q % MR_ROWS, c = 8 * (q / MR_ROWS);
    if (m >= p.M || n0 + c >= p.N) continue;
    const int off = c / 4 * PG_BM + m - mt * PG_BM;
    float4 x[2] = {__ldcg(first + off), __ldcg(first + off + PG_BM)};
#pragma unroll 2
    for (int k = c0 + 1; k <= c1; ++k) {  // the tile is the first of every further pair's share
      const float4* src = rest + static_cast<int64_t>(2 * k) * (PG_BM * PG_BN / 4) + off;
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const float4 y = __ldcg(src + u * PG_BM);
        x[u].x += y.x, x[u].y += y.y, x[u].z += y.z, x[u].w += y.w;
      }
    }
    const int64_t to = static_cast<int64_t>(v.perm[m]) * p.ld_out + n0 + c;
    if (p.out_bf16) {
      *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.out) + to) =
          make_uint4(pack_bf16x2(x[0].x, x[0].y), pack_bf16x2(x[0].z, x[0].w), pack_bf16x2(x[1].x, x[1].y),
                     pack_bf16x2(x[1].z, x[1].w));
    } else {
      float4* out = reinterpret_cast<float4*>(static_cast<float*>(p.out) + to);
      out[0] = x[0], out[1] = x[1];
    }
    const float all[8] = {x[0].x, x[0].y, x[0].z, x[0].w, x[1].x, x[1].y, x[1].z, x[1].w};
    if (!all_finite<8>(all)) multi_repair<kBwd>(mp, v, m, n0 + c, 8);
  }
}

// ====================================================================== gradients of the factors

// dL1[a] = X_a^T (s U_a) and dL2[a]^T = dY_a^T (s T_a) over the rows of group a:
// D is 128 rows of h (or o) by 64 ranks, K runs over the group's 64-row blocks
// of the sorted order, A from X (or dY) as it lies (M-major), B the slots' three
// bf16 parts side by side (N-major, N = 192, each part in accumulator columns of
// its own).  The slots are zero in the rows of a block that belong to others.
// Persistent, one CTA an SM: one thread loads (5 stages of 40 KB), one issues the
// MMAs, four warps add the accumulators to their registers in fp32 after every
// MD_CHAIN blocks (two accumulators, so that the MMAs go on) and store a finished
// tile.  The chain is short because the tensor core cuts its running sum to fp32
// at every step: error of dL2 against 64 bits, 4096 tokens in 4 groups, 2e-6 with
// a group in one chain, 4e-7 so (an fp32 product's is 7e-7).  One CTA for each
// tile and group spent most of its time on the start and end of CTAs with two
// stages: the whole backward took 173 us there and 1065 us for 8190 tokens, 5120 x
// 13824, with it, and takes 167 and 1023 us so.
// When the tiles are fewer than the SMs a group's blocks are dealt to `split`
// items, whose sums go to the partial buffer and are added in order by the one
// that ends last (each epilogue warp its own rows).  No sum depends on timing; adapters without tokens get zeros.
constexpr int MD_BM = 128;
constexpr int MD_BN = 64;
constexpr int MD_BK = 64;
constexpr int MD_THREADS = 192;
constexpr int MD_PARTS = 3;
constexpr int MD_CHAIN = 8;
constexpr int MD_STAGES = 5;
constexpr int MD_A_BYTES = MD_BM * MD_BK * 2;
constexpr int MD_B_BYTES = MD_BN * MD_BK * 2;
constexpr int MD_STAGE_BYTES = MD_A_BYTES + MD_PARTS * MD_B_BYTES;
constexpr int MD_SMEM = MD_STAGES * MD_STAGE_BYTES + 1024 + 256;
constexpr uint32_t MD_TMEM_COLS = 512;  // two accumulators of 192, 256 apart

struct MultiGradSide {
  const uint16_t* A;      // X or dY, batch order
  const uint16_t* slots;  // of U or T
  float* out;             // dL1 [n][h][r] or dL2 [n][r][o]
  int rows;               // h or o
};

struct MultiGradParams {
  MultiGradSide side[2];
  int r, rp, n;
  int tiles0;          // 128-row tiles of dL1, times the rank tiles
  int tiles;           // and of dL2
  int split;           // parts of a group's blocks
  float* partial;      // [group][tile][part] sums of [64][128]
  unsigned* counters;  // [group][tile][epilogue warp], zero at launch
};

// Replaces what is not finite among the `ranks` elements (a multiple of 8) of row m of a factor's
// gradient, from rank j0 on, that this thread has stored at out (`ld` apart) by the sum over the group's
// own tokens with the whole values of U or T, in fp32, eight ranks at a time, up to where all of them
// are NaN.  Never inlined: the path is rare and long.
__device__ __noinline__ void grad_repair(const MultiGradSide& side, const PlanView& v, int grp, int rp, int m, int j0,
                                         int ranks, float* out, int64_t ld) {
  const PlanGroup pg = plan_load(v.groups + grp);
  const int64_t slot0 = pg.slot0 - pg.start / MP_SLOT_ROWS;
  for (int t = 0; t < ranks; t += 8) {
    unsigned bad = 0;
    for (int c = 0; c < 8; ++c)
      if (!isfinite(out[(t + c) * ld])) bad |= 1u << c;
    if (bad == 0) continue;
    float x[8] = {};
#pragma unroll 4
    for (int row = pg.start; row < pg.end; ++row) {
      if ((row - pg.start) % 64 == 63) {
        bool ended = true;
#pragma unroll
        for (int c = 0; c < 8; ++c) ended = ended && (isnan(x[c]) || !(bad >> c & 1));
        if (ended) break;
      }
      const int64_t slot_row = (slot0 + row / MP_SLOT_ROWS) * MP_SLOT_ROWS + row % MP_SLOT_ROWS;
      const uint16_t* b = side.slots + slot_row * (MD_PARTS * rp) + j0 + t;
      const uint4 hi = *reinterpret_cast<const uint4*>(b), mid = *reinterpret_cast<const uint4*>(b + rp),
                  lo = *reinterpret_cast<const uint4*>(b + 2 * rp);
      float w[8] = {};  // the sum of the parts
      axpy8(1.0f, hi, w);
      axpy8(1.0f, mid, w);
      axpy8(1.0f, lo, w);
      const float a = bf16_bits_to_float(side.A[static_cast<int64_t>(v.perm[row]) * side.rows + m]);
#pragma unroll
      for (int c = 0; c < 8; ++c) x[c] = fmaf(a, w[c], x[c]);
    }
#pragma unroll
    for (int c = 0; c < 8; ++c)
      if (bad >> c & 1) out[(t + c) * ld] = x[c];
  }
}

__global__ void __launch_bounds__(MD_THREADS, 1)
    multi_grad_kernel(const __grid_constant__ CUtensorMap tmX, const __grid_constant__ CUtensorMap tmXs,
                      const __grid_constant__ CUtensorMap tmD, const __grid_constant__ CUtensorMap tmDs,
                      const __grid_constant__ CUtensorMap tmU, const __grid_constant__ CUtensorMap tmT,
                      const __grid_constant__ MultiGradParams p, const __grid_constant__ PlanView v) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + MD_STAGES * MD_STAGE_BYTES);
  uint64_t* empty = full + MD_STAGES;
  uint64_t* tfull = empty + MD_STAGES;
  uint64_t* tempty = tfull + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(tempty + 2);

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int n_tiles = p.rp / MD_BN;
  const int64_t items = static_cast<int64_t>(p.tiles) * p.n * p.split;
  // item u: part u % split of tile (u / split) % tiles of an adapter, so that an SM's items
  // are of different adapters
  struct Item {
    int second, m0, j0, adapter, grp;
    int tile, part;
    int i0, blocks;  // 64-row blocks i0 .. i0 + blocks - 1 of the sorted order
    PlanGroup pg;
  };
  auto item_of = [&](int64_t u) -> Item {
    Item it{};
    const int part = static_cast<int>(u % p.split);
    const int64_t w = u / p.split;
    it.adapter = static_cast<int>(w / p.tiles);
    int tile = static_cast<int>(w - static_cast<int64_t>(it.adapter) * p.tiles);
    it.tile = tile;
    it.part = part;
    it.second = tile >= p.tiles0 ? 1 : 0;
    if (it.second) tile -= p.tiles0;
    it.m0 = (tile / n_tiles) * MD_BM;
    it.j0 = (tile % n_tiles) * MD_BN;
    it.grp = __ldg(v.adp_group + it.adapter);
    if (it.grp >= 0) {
      it.pg = plan_load(v.groups + it.grp);
      const int b0 = it.pg.start / MD_BK, b = (it.pg.end - 1) / MD_BK - b0 + 1;
      it.i0 = b0 + b * part / p.split;
      it.blocks = b0 + b * (part + 1) / p.split - it.i0;
    }
    return it;
  };

  if (threadIdx.x == 0) {
    for (int s = 0; s < MD_STAGES; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&tfull[b], 1);
      mbar_init(&tempty[b], 4);
    }
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, MD_TMEM_COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  pdl_launch_dependents();
  pdl_wait();

  if (warp == 0) {
    if (lane == 0) {
      const bool in_order = v.head->in_order != 0;
      int G = 0;
      bool ok = true;
      for (int64_t u = blockIdx.x; u < items && ok; u += gridDim.x) {
        const Item it = item_of(u);
        const CUtensorMap* ma = it.second ? (in_order ? &tmD : &tmDs) : (in_order ? &tmX : &tmXs);
        const CUtensorMap* mb = it.second ? &tmT : &tmU;
        for (int i = 0; i < it.blocks; ++i, ++G) {
          const int s = G % MD_STAGES;
          if (!mbar_wait(&empty[s], ((G / MD_STAGES) & 1) ^ 1)) {
            ok = false;
            break;
          }
          uint8_t* st = smem + s * MD_STAGE_BYTES;
          const int row = (it.i0 + i) * MD_BK;
          // the block's rows within the group's slots
          const int y = (it.pg.slot0 + row / MP_SLOT_ROWS - it.pg.start / MP_SLOT_ROWS) * MP_SLOT_ROWS + row % MP_SLOT_ROWS;
          mbar_arrive_expect_tx(&full[s], MD_STAGE_BYTES);
          tma_load_2d(st, ma, &full[s], it.m0, row);
          tma_load_2d(st + MD_A_BYTES / 2, ma, &full[s], it.m0 + 64, row);
          for (int h = 0; h < MD_PARTS; ++h)
            tma_load_2d(st + MD_A_BYTES + h * MD_B_BYTES, mb, &full[s], h * p.rp + it.j0, y);
        }
      }
      for (int g = G - MD_STAGES > 0 ? G - MD_STAGES : 0; g < G; ++g) mbar_wait(&full[g % MD_STAGES], (g / MD_STAGES) & 1);
    }
  } else if (warp == 1) {
    if (lane == 0) {
      const uint32_t idesc = idesc_bf16(MD_BM, MD_PARTS * MD_BN, true, true);
      int G = 0, C = 0;  // stages and chains so far
      bool ok = true;
      for (int64_t u = blockIdx.x; u < items && ok; u += gridDim.x) {
        const Item it = item_of(u);
        for (int c = 0; c < it.blocks && ok; c += MD_CHAIN, ++C) {
          if (!mbar_wait(&tempty[C & 1], ((C >> 1) & 1) ^ 1)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const int end = min(it.blocks, c + MD_CHAIN);
          for (int i = c; i < end; ++i, ++G) {
            const int s = G % MD_STAGES;
            if (!mbar_wait(&full[s], (G / MD_STAGES) & 1)) {
              ok = false;
              break;
            }
            tc_fence_after();
            const uint32_t a_base = smem_u32(smem + s * MD_STAGE_BYTES);
#pragma unroll
            for (int kk = 0; kk < MD_BK / 16; ++kk)
              umma_bf16(tmem + 256u * (C & 1), sw128_desc(a_base + kk * 2048, MD_A_BYTES / 2, 1024),
                        sw128_desc(a_base + MD_A_BYTES + kk * 2048, MD_B_BYTES, 1024), idesc, (i > c || kk > 0) ? 1u : 0u);
            umma_commit(&empty[s]);
          }
          if (ok) umma_commit(&tfull[C & 1]);
        }
      }
    }
  } else {
    // ---------------- epilogue: thread = row of the tile
    const int q = warp & 3;  // TMEM lanes 32 q .. 32 q + 31
    const int row = 32 * q + lane;
    int C = 0;
    bool ok = true;
    for (int64_t u = blockIdx.x; u < items && ok; u += gridDim.x) {
      const Item it = item_of(u);
      const MultiGradSide& side = p.side[it.second];
      float x[MD_BN];
#pragma unroll
      for (int j = 0; j < MD_BN; ++j) x[j] = 0.0f;
      for (int c = 0; c < it.blocks; c += MD_CHAIN, ++C) {
        if (!__all_sync(0xFFFFFFFFu, mbar_wait(&tfull[C & 1], (C >> 1) & 1))) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t at = tmem + (static_cast<uint32_t>(q * 32) << 16) + 256u * (C & 1);
#pragma unroll
        for (int h = MD_PARTS - 1; h >= 0; --h)
#pragma unroll
          for (int k = 0; k < MD_BN; k += 16) {
            uint32_t r[16];
            tmem_ld16(at + h * MD_BN + k, r);
            tmem_ld_wait();
#pragma unroll
            for (int t = 0; t < 16; ++t) x[k + t] += __uint_as_float(r[t]);
          }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&tempty[C & 1]);
      }
      if (!ok) break;
      if (it.grp < 0 && it.part > 0) continue;  // zeros are stored once
      if (p.split > 1 && it.grp >= 0) {
        const int64_t tile_index = static_cast<int64_t>(it.grp) * p.tiles + it.tile;
        float* part = p.partial + (tile_index * p.split + it.part) * (MD_BM * MD_BN) + row;  // [rank][row]: coalesced
#pragma unroll
        for (int j = 0; j < MD_BN; ++j) part[j * MD_BM] = x[j];
        // by warp, each for its own 32 rows: a barrier of the four would wait for good where one gave up
        __threadfence();
        __syncwarp();
        unsigned prior = 0;
        if (lane == 0) prior = atomicAdd(&p.counters[tile_index * 4 + q], 1u);
        prior = __shfl_sync(0xFFFFFFFFu, prior, 0);
        if (prior != static_cast<unsigned>(p.split - 1)) continue;
        __threadfence();
        const float* first = p.partial + tile_index * p.split * (MD_BM * MD_BN) + row;
#pragma unroll
        for (int j = 0; j < MD_BN; ++j) x[j] = __ldcg(first + j * MD_BM);
        for (int k = 1; k < p.split; ++k)
#pragma unroll
          for (int j = 0; j < MD_BN; ++j) x[j] += __ldcg(first + (k * MD_BN + j) * MD_BM);
      }
      const int m = it.m0 + row;
      if (m >= side.rows) continue;
      float* out = side.out + static_cast<int64_t>(it.adapter) * p.r * side.rows;
      const int ranks = min(MD_BN, p.r - it.j0);
      if (it.second) {
#pragma unroll
        for (int j = 0; j < MD_BN; ++j)
          if (j < ranks) out[static_cast<int64_t>(it.j0 + j) * side.rows + m] = x[j];
      } else {
        float4* dst = reinterpret_cast<float4*>(out + static_cast<int64_t>(m) * p.r + it.j0);
#pragma unroll
        for (int j = 0; j < MD_BN; j += 4)
          if (j < ranks) dst[j / 4] = make_float4(x[j], x[j + 1], x[j + 2], x[j + 3]);
      }
      if (it.grp >= 0 && !all_finite<MD_BN>(x)) {
        if (it.second)
          grad_repair(side, v, it.grp, p.rp, m, it.j0, ranks, out + static_cast<int64_t>(it.j0) * side.rows + m, side.rows);
        else
          grad_repair(side, v, it.grp, p.rp, m, it.j0, ranks, out + static_cast<int64_t>(m) * p.r + it.j0, 1);
      }
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, MD_TMEM_COLS);
  }
}

}  // namespace qlora
