// lora.cu -- low-rank adapters of many requests beside one FP4 projection: all
// that is not the projection itself (project.cu, rows.cu).
//
//   forward   V = scale_i X A_i^T,  Y = X W^T + V B_i^T
//   backward  U = scale_i dY B_i,   dX = dY W + U A_i,  dA_i = sum_t U^T X,
//             dB_i = sum_t dY^T V
// with i the adapter of the row's request.  Requests are runs of rows
// [seg_ptr[s], seg_ptr[s+1]) whose number is known to the host and whose
// lengths are not: grids are sized by bounds, and a block finds its request by
// comparing every request's range at once (one round of independent loads).
// All of it is memory-bound: X and dY are read once by each product, 2 bytes an
// element for 2 rank operations.
// V and U are summed in FP32 and kept so; as operands of a BF16 product (tiles
// of 256 rows, gradients) they are two BF16 terms, 16 bits of the value.
#include "lowrank.cuh"
#include "tile.cuh"

namespace nvfp4 {

namespace {

// A request's rows, clamped to the batch so that no index leaves it.
struct Rows { int begin, end; };
__device__ __forceinline__ Rows request_rows(const int* __restrict__ seg_ptr, int s, int T) {
  const int b = min(max(__ldg(seg_ptr + s), 0), T), e = min(max(__ldg(seg_ptr + s + 1), b), T);
  return Rows{b, e};
}

// The request whose blocks of `span` rows, counted from its first row, include
// block `w` of the launch: blocks of request s have numbers begin / span + s
// .. (unique, as ceil(len / span) <= floor(end / span) - floor(begin / span) +
// 1).  Returns it in *req (-1: none) and its block in *blk.  Block-wide.  Where
// ranges that decrease make several requests claim a block, the last of them has
// it: the same one in every CTA of a cluster, and a block that it has.
__device__ __forceinline__ void find_block(const int* __restrict__ seg_ptr, int S, int T, int span, int w, int* sh, int* req,
                                           int* blk) {
  if (threadIdx.x == 0) sh[0] = -1;
  __syncthreads();
  for (int s = threadIdx.x; s < S; s += blockDim.x) {
    const Rows r = request_rows(seg_ptr, s, T);
    const int first = r.begin / span + s, n = (r.end - r.begin + span - 1) / span;
    if (w >= first && w < first + n) atomicMax(sh, s);
  }
  __syncthreads();
  *req = sh[0];
  *blk = sh[0] < 0 ? 0 : w - (request_rows(seg_ptr, sh[0], T).begin / span + sh[0]);
}

__device__ __forceinline__ int checked_adapter(const int* __restrict__ seg_adapter, int s, int count) {
  const int id = __ldg(seg_adapter + s);
  return id >= 0 && id < count ? id : -1;
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool ok) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(ok ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

__device__ __forceinline__ void ldmatrix_x4_trans(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void mma_16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
               "{%0, %1, %2, %3};"
               : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
               : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// 64 columns (128 bytes) of a row in shared memory: 16-byte chunk c of row r
// sits at chunk c ^ (r % 8), so eight rows of one chunk hit distinct banks.
__device__ __forceinline__ uint32_t swz(int row, int chunk) {
  return static_cast<uint32_t>(row * 128 + ((chunk ^ (row & 7)) << 4));
}

// ---------------------------------------------------------------------------
// Plan (last blocks of the shrink launch), one block for each 256-row tile: the
// adapter of each row (-1 none, -2 padding), and the adapters that the tile has
// rows of, each of which costs the tile one K step (0.3 us for 256 x 256).
// `seen`: a bit for each adapter, in shared memory.
// ---------------------------------------------------------------------------
struct PlanOut {
  int* valid_rows;
  int* tile_count;
  int* tile_base;
  int* tile_direct;
  int* slab_adapter;   // or null: no slabs to come
  int* row_adapter;
};

__device__ void plan_tile(const int* __restrict__ seg_ptr, const int* __restrict__ seg_adapter, int S, int T, int count,
                          int tile, const PlanOut& out, uint32_t* seen, int* sh) {
  const int words = (count + 31) / 32, t0 = tile * 256;
  if (threadIdx.x < 2) sh[threadIdx.x] = 0;
  for (int w = threadIdx.x; w < words; w += blockDim.x) seen[w] = 0u;
  const int valid = S > 0 ? min(max(__ldg(seg_ptr + S), 0), T) : 0;
  for (int t = t0 + threadIdx.x; t < min(t0 + 256, T); t += blockDim.x) out.row_adapter[t] = t < valid ? -1 : -2;
  if (tile == 0 && threadIdx.x == 0) *out.valid_rows = valid;
  __syncthreads();
  for (int s = threadIdx.x; s < S; s += blockDim.x) {
    const Rows r = request_rows(seg_ptr, s, T);
    if (r.end <= t0) atomicAdd(&sh[0], 1);
    const int id = checked_adapter(seg_adapter, s, count), b = max(r.begin, t0), e = min(r.end, t0 + 256);
    if (id >= 0 && b < e) {
      atomicOr(&seen[id >> 5], 1u << (id & 31));
      for (int t = b; t < e; ++t) out.row_adapter[t] = id;
    }
  }
  __syncthreads();
  if (!out.slab_adapter) return;
  if (threadIdx.x < 32) {   // the adapters in ascending order
    // requests before the tile + tiles before it: the tile's slabs fit between
    // this and the next tile's base (no more adapters than requests; a request
    // that reaches into the next tile is counted there again, and there is one
    // more tile)
    const int base = sh[0] + tile;
    int n = 0;
    for (int w0 = 0; w0 < words; w0 += 32) {
      const int w = w0 + threadIdx.x;
      uint32_t bits = w < words ? seen[w] : 0u;
      int at = __popc(bits);
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int up = __shfl_up_sync(0xFFFFFFFFu, at, o);
        if (static_cast<int>(threadIdx.x) >= o) at += up;
      }
      const int total = __shfl_sync(0xFFFFFFFFu, at, 31);
      at += n - __popc(bits);
      for (; bits; bits &= bits - 1) out.slab_adapter[base + at++] = 32 * w + __ffs(bits) - 1;
      n += total;
    }
    if (threadIdx.x == 0) {
      out.tile_base[tile] = base;
      out.tile_count[tile] = n;
      out.tile_direct[tile] = 0;   // slab_part may set it
    }
  }
}

// The largest magnitude (BF16 bits) in the second operand of an adapter, one
// block for each of `parts` parts of an adapter some request uses.  Where it is
// not finite slab_part keeps the adapter out: in a tile that adapters share, the
// other adapters' rows are zeros in this one's slab, and 0 x NaN would reach them.
__device__ void second_maximum(const uint16_t* E, int64_t elements, const int* __restrict__ seg_adapter, int S,
                               int id, int part, int parts, int* __restrict__ second_max, int* sh) {
  if (threadIdx.x < 2) sh[threadIdx.x] = 0;
  __syncthreads();
  for (int s = threadIdx.x; s < S; s += blockDim.x)
    if (__ldg(seg_adapter + s) == id) sh[0] = 1;
  __syncthreads();
  if (!sh[0]) return;
  const uint4* v = reinterpret_cast<const uint4*>(E + id * elements);
  const int64_t n8 = elements / 8, lo = n8 * part / parts, hi = n8 * (part + 1) / parts;
  uint32_t m = 0;
#pragma unroll 8
  for (int64_t i = lo + threadIdx.x; i < hi; i += blockDim.x) m = max(m, absmax_bits8(v[i]));
  m = __reduce_max_sync(0xFFFFFFFFu, m);
  if ((threadIdx.x & 31) == 0) atomicMax(&sh[1], static_cast<int>(m));
  __syncthreads();
  if (threadIdx.x == 0) second_max[id * kCheckParts + part] = sh[1];
}

// ---------------------------------------------------------------------------
// V[t, j] = scale_i sum_c x[t, c] A_i[j, c].  Work item: 128 rows of a request; a cluster
// of `slices` CTAs splits the sum over c and adds its parts in CTA order.  On
// the 5th-generation tensor core (M = 128, N = rank, K = 16 a step), as
// mma.sync needed 60 us for the 2 x 8192 x 8192 x 64 operations that read
// memory for 21 (this form: 37 from a cold start, 31 within a sequence).
//   warp 0    TMA: x [128 x 64] and A [rank x 64] tiles into the ring;
//   warp 1    MMA issuer;
//   warps 2-5 max |x| over the request's rows (of any adapter or none) from
//             the tiles on their way (the quantizer's first pass over x costs
//             a launch and a read otherwise); then the epilogue:
//             partial sums are stored into the CTA of the cluster that adds
//             them, through distributed shared memory.
// ---------------------------------------------------------------------------
constexpr int kShrinkRows = 128, kShrinkThreads = 192, kShrinkMaxStages = 6;
constexpr uint32_t kShrinkRing = 73 * 1024;   // three CTAs an SM

struct ShrinkParams {
  int T, K, count, rank, n_pad;   // n_pad: rank rounded up to 16, the MMA's N
  int stages, slices, S, items, plan_tiles;   // items: clusters that may have work
  const float* scale;
  const int* seg_ptr;
  const int* seg_adapter;
  PlanOut plan;
  const uint16_t* E;     // second operands whose maxima are taken, or null
  int64_t elements;
  int parts;
  int* second_max;
  unsigned int* amax;
  float* V;
  bool after;   // A comes from the launch before
};

__global__ void __launch_bounds__(kShrinkThreads)
lora_shrink_kernel(const __grid_constant__ CUtensorMap tmX, const __grid_constant__ CUtensorMap tmX32,
                   const __grid_constant__ CUtensorMap tmA,
                   const __grid_constant__ ShrinkParams p) {
  extern __shared__ uint8_t dyn[];
  allow_next_kernel();
  if (p.after) wait_previous_kernel();
  // Every CTA waits for the launch before it ends, whatever it finds to do: the
  // launch after this one waits for this one only, and reads what that one zeroes.
  __shared__ int sh[2];
  __shared__ uint64_t full[kShrinkMaxStages], empty[kShrinkMaxStages], acc_full;
  __shared__ uint32_t tmem_slot;
  const int slices = p.slices, slice = slices > 1 ? static_cast<int>(cluster_ctarank()) : 0;
  const int item = blockIdx.x / slices;
  // the last CTAs make the plan's tiles and the checks, one each; these and every
  // return below are uniform over the cluster
  if (item >= p.items) {
    const int unit = static_cast<int>(blockIdx.x) - p.items * slices;
    if (unit < p.plan_tiles)
      plan_tile(p.seg_ptr, p.seg_adapter, p.S, p.T, p.count, unit, p.plan, reinterpret_cast<uint32_t*>(dyn), sh);
    else if (p.E && unit - p.plan_tiles < p.count * p.parts)
      second_maximum(p.E, p.elements, p.seg_adapter, p.S, (unit - p.plan_tiles) / p.parts, (unit - p.plan_tiles) % p.parts,
                   p.parts, p.second_max, sh);
    wait_previous_kernel();
    return;
  }
  int s, blk;
  find_block(p.seg_ptr, p.S, p.T, kShrinkRows, item, sh, &s, &blk);
  if (s < 0) {
    wait_previous_kernel();
    return;
  }
  const int id = checked_adapter(p.seg_adapter, s, p.count);
  const Rows req = request_rows(p.seg_ptr, s, p.T);
  const int t0 = req.begin + blk * kShrinkRows, n = min(kShrinkRows, req.end - t0);
  const int chunks = p.K / 64, c0 = chunks * slice / slices, nc = chunks * (slice + 1) / slices - c0;
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(dyn) + 1023) & ~uintptr_t(1023));
  constexpr uint32_t X_TILE = kShrinkRows * 128;
  const uint32_t stage_bytes = X_TILE + p.n_pad * 128;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    for (int i = 0; i < p.stages; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 5);   // the MMAs' commit and four warps
    }
    mbar_init(&acc_full, 1);
    fence_barrier_init();
    prefetch_tmap(&tmX);
    prefetch_tmap(&tmA);
  }
  if (warp == 1) tmem_alloc(&tmem_slot, 128);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_slot;
  if (warp == 0 && lane == 0) {
    // a short request loads boxes of 32 rows, not 128 (the tile's other rows are
    // whatever the ring held, and so are the sums of rows that do not exist)
    const int boxes = (n + 31) / 32;
    int stage = 0, last = 0;
    uint32_t phase = 0;
    for (int i = 0; i < nc; ++i) {
      if (!mbar_wait(&empty[stage], phase ^ 1u, kErrWaitEmpty)) break;
      mbar_arrive_expect_tx(&full[stage], boxes * (X_TILE / 4) + (id >= 0 ? p.n_pad * 128 : 0));
      if (boxes == 4)
        tma_load_2d(smem + stage * stage_bytes, &tmX, &full[stage], (c0 + i) * 64, t0);
      else
        for (int k = 0; k < boxes; ++k)
          tma_load_2d(smem + stage * stage_bytes + k * (X_TILE / 4), &tmX32, &full[stage], (c0 + i) * 64, t0 + 32 * k);
      if (id >= 0) tma_load_2d(smem + stage * stage_bytes + X_TILE, &tmA, &full[stage], (c0 + i) * 64, id * p.rank);
      last = i + 1;
      if (++stage == p.stages) stage = 0, phase ^= 1u;
    }
    for (int i = max(0, last - p.stages); i < last; ++i)
      mbar_wait(&full[i % p.stages], static_cast<uint32_t>(i / p.stages) & 1u, kErrWaitFull);
  } else if (warp == 1 && lane == 0) {
    const uint32_t idesc = (1u << 4) | (1u << 7) | (1u << 10) | (static_cast<uint32_t>(p.n_pad >> 3) << 17) | (8u << 24);
    int stage = 0;
    uint32_t phase = 0;
    for (int i = 0; i < nc; ++i) {
      if (!mbar_wait(&full[stage], phase, kErrWaitFull)) break;
      tc_fence_after();
      if (id >= 0) {
        const uint32_t at = smem_u32(smem + stage * stage_bytes);
        const uint64_t adesc = smem_desc(at, 16, 1024, 2), bdesc = smem_desc(at + X_TILE, 16, 1024, 2);
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) mma_bf16(tmem, adesc + 2 * kk, bdesc + 2 * kk, idesc, (i | kk) != 0);
        tc_commit(&empty[stage]);
      } else {
        mbar_arrive(&empty[stage]);
      }
      if (++stage == p.stages) stage = 0, phase ^= 1u;
    }
    if (id >= 0)
      tc_commit(&acc_full);
    else
      mbar_arrive(&acc_full);
    mbar_wait(&acc_full, 0, kErrWaitAccFull);
  } else if (warp >= 2) {
    // a row of the tile is 128 bytes, in an order that the swizzle permutes
    // within the row only: a thread takes a row
    uint32_t m = 0;
    int stage = 0;
    uint32_t phase = 0;
    const int row = tid - 64;
    for (int i = 0; i < nc; ++i) {
      if (!mbar_wait(&full[stage], phase, kErrWaitFull)) break;
      if (row < n) {
        const uint4* x = reinterpret_cast<const uint4*>(smem + stage * stage_bytes + row * 128);
        uint4 v[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] = x[(k + row) & 7];   // neighbours on distinct banks
        uint32_t m2 = 0;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          m2 = __vmaxu2(m2, __vmaxu2(v[k].x & 0x7FFF7FFFu, v[k].y & 0x7FFF7FFFu));
          m2 = __vmaxu2(m2, __vmaxu2(v[k].z & 0x7FFF7FFFu, v[k].w & 0x7FFF7FFFu));
        }
        m = max(m, max(m2 & 0xFFFFu, m2 >> 16));
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&empty[stage]);
      if (++stage == p.stages) stage = 0, phase ^= 1u;
    }
    m = __reduce_max_sync(0xFFFFFFFFu, m);
    wait_previous_kernel();   // *amax is zero
    if (lane == 0 && m) atomicMax(p.amax, m << 16);
  }
  __syncwarp();
  if (warp >= 2) mbar_wait(&acc_full, 0, kErrWaitAccFull);
  __syncwarp();
  // part[q][i][n_pad]: slice q's sums of row slice + slices i
  float* part = reinterpret_cast<float*>(smem);
  const int mine = kShrinkRows / slices, shift = 31 - __clz(slices);
  if (id >= 0) {
    if (slices > 1)   // every reader of the ring (in every CTA) is done
      cluster_sync();
    else
      __syncthreads();
    if (warp >= 2) {
      tc_fence_after();
      const int r = (warp & 3) * 32 + lane;
      const uint32_t to = mapa_shared(smem_u32(part) + (slice * mine + (r >> shift)) * p.n_pad * 4, r & (slices - 1));
      for (int c = 0; c < p.n_pad; c += 32) {
        uint32_t v[32];
        tmem_ld_32x32b_x32(tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16) + c, v);
        tmem_ld_wait();
#pragma unroll
        for (int e = 0; e < 32; e += 4)
          if (c + e < p.n_pad)
            asm volatile("st.shared::cluster.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(to + (c + e) * 4), "r"(v[e]), "r"(v[e + 1]),
                         "r"(v[e + 2]), "r"(v[e + 3])
                         : "memory");
      }
    }
    tc_fence_before();
    if (slices > 1) cluster_sync();
  }
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, 128);
  if (id < 0) return;
  const float sc = __ldg(p.scale + id);
  const int words = p.rank / 4;
  for (int u = tid; u < mine * words; u += kShrinkThreads) {
    const int i = u / words, j = (u - i * words) * 4, r = slice + slices * i;
    if (r >= n) continue;
    float4 sum = *reinterpret_cast<const float4*>(part + i * p.n_pad + j);
    for (int q = 1; q < slices; ++q) {
      const float4 v = *reinterpret_cast<const float4*>(part + (q * mine + i) * p.n_pad + j);
      sum.x += v.x;
      sum.y += v.y;
      sum.z += v.z;
      sum.w += v.w;
    }
    *reinterpret_cast<float4*>(p.V + static_cast<int64_t>(t0 + r) * p.rank + j) =
        make_float4(sum.x * sc, sum.y * sc, sum.z * sc, sum.w * sc);
  }
}

// The same for many short requests (a 128-row item of a single row costs what a
// full one does): a block for each row and eight ranks.  Then the plan's tiles
// and the checks, as above.
__global__ void __launch_bounds__(kRowThreads) lora_shrink_rows_kernel(const uint16_t* __restrict__ x, int64_t ldx,
                                                                       const uint16_t* A,
                                                                       const __grid_constant__ ShrinkParams p) {
  extern __shared__ uint8_t dyn[];
  __shared__ int sh[2], row_id;
  __shared__ RowSums sums;
  allow_next_kernel();
  if (p.after) wait_previous_kernel();
  const int groups = p.rank / 8, unit = static_cast<int>(blockIdx.x) - p.T * groups;
  if (unit >= 0) {
    if (unit < p.plan_tiles)
      plan_tile(p.seg_ptr, p.seg_adapter, p.S, p.T, p.count, unit, p.plan, reinterpret_cast<uint32_t*>(dyn), sh);
    else
      second_maximum(p.E, p.elements, p.seg_adapter, p.S, (unit - p.plan_tiles) / p.parts, (unit - p.plan_tiles) % p.parts,
                   p.parts, p.second_max, sh);
    wait_previous_kernel();   // as every block (see above)
    return;
  }
  const int t = blockIdx.x / groups, grp = blockIdx.x - t * groups;
  const bool live = t < max(__ldg(p.seg_ptr + p.S), 0);
  const int id = live ? row_adapter_of(p.seg_ptr, p.seg_adapter, p.S, p.count, t, &row_id) : -1;
  unsigned int* amax = grp == 0 ? p.amax : nullptr;
  if (!live || (id < 0 && !amax)) {
    wait_previous_kernel();
    return;
  }
  const int at = max(id, 0);
  row_low_rank(x + t * ldx, id >= 0 ? A + (static_cast<int64_t>(id) * p.rank + grp * 8) * p.K : nullptr, p.K, p.scale + at,
               p.V + static_cast<int64_t>(t) * p.rank + grp * 8, amax, sums);
}

// The rows of adapter `id`, in order, from sorted[span[id].x] on (span[id].y of
// them): after those of the adapters before it.  Block-wide, 256 threads.  Rows
// of a seg_ptr that is out of order may be missing; no index leaves the batch.
__device__ __forceinline__ void list_rows(const LoraBatch& b, int T, int id, int* __restrict__ sorted, int2* __restrict__ span) {
  __shared__ int begin[256], upto[257];
  __shared__ unsigned int warps[2][8];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  unsigned int before = 0, own = 0;
  int id_of = -1;   // of the thread's request in the chunk
  Rows mine = {0, 0};
  for (int s = tid; s < b.S; s += 256) {
    id_of = checked_adapter(b.seg_adapter, s, b.count);
    mine = request_rows(b.seg_ptr, s, T);
    if (id_of >= 0 && id_of < id) before += mine.end - mine.begin;
    if (id_of == id) own += mine.end - mine.begin;
  }
  before = __reduce_add_sync(0xFFFFFFFFu, before);
  own = __reduce_add_sync(0xFFFFFFFFu, own);
  if (lane == 0) warps[0][warp] = before, warps[1][warp] = own;
  __syncthreads();
  before = own = 0;
#pragma unroll
  for (int w = 0; w < 8; ++w) before += warps[0][w], own += warps[1][w];
  const int first = static_cast<int>(min(before, static_cast<unsigned int>(T)));
  const int n = static_cast<int>(min(own, static_cast<unsigned int>(T - first)));
  if (tid == 0) span[id] = make_int2(first, n);
  for (int c = 0, done = 0; c < b.S && done < n; c += 256) {
    if (b.S > 256) {
      id_of = c + tid < b.S ? checked_adapter(b.seg_adapter, c + tid, b.count) : -1;
      if (id_of == id) mine = request_rows(b.seg_ptr, c + tid, T);
    }
    const int len = id_of == id ? mine.end - mine.begin : 0;
    unsigned int sum = len;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const unsigned int v = __shfl_up_sync(0xFFFFFFFFu, sum, o);
      if (lane >= o) sum += v;
    }
    __syncthreads();   // the sums above, or the last chunk's lists, are read
    begin[tid] = mine.begin;
    if (lane == 31) warps[0][warp] = sum;
    if (tid == 0) upto[0] = 0;
    __syncthreads();
    for (int w = 0; w < warp; ++w) sum += warps[0][w];
    upto[tid + 1] = static_cast<int>(min(sum, 1u << 30));
    __syncthreads();
    const int total = min(upto[256], n - done);
    for (int r = tid; r < total; r += 256) {
      int k = 0;   // the last request with upto[k] <= r: it has the row
#pragma unroll
      for (int o = 128; o > 0; o >>= 1)
        if (upto[k + o] <= r) k += o;
      sorted[first + done + r] = min(max(begin[k] + r - upto[k], 0), T - 1);
    }
    done += total;
  }
}

// ---------------------------------------------------------------------------
// A [count][rank][Cin] -> [count][Cin][rank] and B [count][Cout][rank] ->
// [count][rank][Cout] in 64 x 32 tiles (rank along the 32).  Also zeroes *amax, and
// one block for each adapter lists its rows.
// ---------------------------------------------------------------------------
__global__ void __launch_bounds__(256) transpose_kernel(const uint16_t* __restrict__ A, uint16_t* __restrict__ a_t, int Cin,
                                                        const uint16_t* __restrict__ B, uint16_t* __restrict__ b_t, int Cout,
                                                        int rank, float* __restrict__ amax, const LoraBatch b, int T,
                                                        int* __restrict__ sorted, int2* __restrict__ span) {
  allow_next_kernel();
  if (blockIdx.x == 0) {
    if (blockIdx.y == 0) list_rows(b, T, blockIdx.z, sorted, span);
    return;
  }
  __shared__ uint16_t tile[64][34];
  const int block = blockIdx.x - 1;
  const bool second = block >= Cin / 64;
  const int C = second ? Cout : Cin, c0 = (block - (second ? Cin / 64 : 0)) * 64, j0 = blockIdx.y * 32;
  const int64_t base = static_cast<int64_t>(blockIdx.z) * rank * C;
  if (block == 0 && blockIdx.y == 0 && blockIdx.z == 0 && threadIdx.x == 0) *amax = 0.0f;
  // along c: 64 lanes x 4 ranks a step; along the rank: 32 lanes x 8 channels
  const int cx = threadIdx.x & 63, cj = threadIdx.x >> 6, jx = threadIdx.x & 31, jc = threadIdx.x >> 5;
  if (!second) {
#pragma unroll
    for (int j = cj; j < 32; j += 4)
      if (j0 + j < rank) tile[cx][j] = A[base + static_cast<int64_t>(j0 + j) * C + c0 + cx];
    __syncthreads();
#pragma unroll
    for (int c = jc; c < 64; c += 8)
      if (j0 + jx < rank) a_t[base + static_cast<int64_t>(c0 + c) * rank + j0 + jx] = tile[c][jx];
  } else {
#pragma unroll
    for (int c = jc; c < 64; c += 8)
      if (j0 + jx < rank) tile[c][jx] = B[base + static_cast<int64_t>(c0 + c) * rank + j0 + jx];
    __syncthreads();
#pragma unroll
    for (int j = cj; j < 32; j += 4)
      if (j0 + j < rank) b_t[base + static_cast<int64_t>(j0 + j) * C + c0 + cx] = tile[cx][j];
  }
}

// ---------------------------------------------------------------------------
// G_i[j, c] = sum over the rows t of adapter i of P[t, j] Z[t, c]: dA from U and
// X, dB from V and dY, in one launch.  Block (128 columns c, adapter i) walks the
// adapter's list of rows, 64 a step whatever requests they come from (a step for
// each request's rows: 77 requests of 23 rows, rank 128, 83 us; so 44), both
// operands through a cp.async ring.  With few adapters a cluster of up to eight
// CTAs splits the steps and adds its sums in CTA order (one adapter, 4096 rows,
// 1024 x 1024, rank 32: the whole backward 72 and 41 us).  P is FP32 and enters as
// two BF16 terms, high and low, which keeps 16 bits of it.  Both operands have the
// summed index outermost, so their fragments are read transposed.  An adapter
// without rows gets zeros.  8192 x 5120 x 5120, rank 32, beside the kernels that
// make dX: 73 us for 168 MB (26 at HBM's rate); it shares the SMs with them.
// ---------------------------------------------------------------------------
struct GradSide {
  const float* P;       // [T, rank]
  const uint16_t* z;    // [T, C], pitch ldz
  int64_t ldz;
  int C;
  __nv_bfloat16* G;     // [count][rank][C], or with `transposed` [count][C][rank]
};

template <int MT>   // tiles of 16 ranks
__global__ void __launch_bounds__(128)
lora_grad_kernel(GradSide da, GradSide db, int rank, const int* sorted, const int2* span,
                 int slices) {
  constexpr int STAGES = MT == 8 ? 2 : 3;
  constexpr uint32_t Z_TILE = 2 * 64 * 128,   // two halves of 64 columns
                      P_TILE = 64 * MT * 16 * 4, STAGE = Z_TILE + P_TILE;
  constexpr uint32_t P_PITCH = MT * 32 + 16;   // bytes of a BF16 row of P; 16 more: rows start on different banks
  extern __shared__ __align__(128) uint8_t dyn[];
  const uint32_t base = (smem_u32(dyn) + 127) & ~127u;
  uint8_t* gen = dyn + (base - smem_u32(dyn));
  uint8_t* hi = gen + STAGES * STAGE;
  uint8_t* lo = hi + 64 * P_PITCH;
  wait_previous_kernel();
  const int slice = slices > 1 ? static_cast<int>(cluster_ctarank()) : 0;
  const int block = blockIdx.x / slices, blocks_a = (da.C + 127) / 128;
  const bool transposed = block >= blocks_a;
  const GradSide side = transposed ? db : da;
  const int id = blockIdx.y, col0 = (block - (transposed ? blocks_a : 0)) * 128;
  const bool wide = col0 + 128 <= side.C;   // else the second half of the columns does not exist
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  float acc[MT][4][4] = {};
  const int2 list = span[id];
  // this CTA's steps: those of the list with number slice modulo `slices`
  const int steps = ((list.y + 63) / 64 - slice + slices - 1) / slices;
  auto row0 = [&](int step) { return 64 * (slice + step * slices); };
  // the rows of four steps, from the one under way on
  __shared__ int rows[4][64];
  auto row_of = [&](int step) {
    return step < steps && row0(step) + tid < list.y ? sorted[list.x + row0(step) + tid] : 0;
  };
  if (tid < 64)
#pragma unroll
    for (int i = 0; i < 4; ++i) rows[i][tid] = row_of(i);
  __syncthreads();
  int later = tid < 64 ? row_of(4) : 0;
  const uint16_t* z = side.z + col0 + (tid & 7) * 8;
  auto load = [&](int step, int stage) {
    const uint32_t at = base + stage * STAGE;
    const int* row = rows[step & 3];
    const int n = list.y - row0(step);
#pragma unroll
    for (int r = tid >> 3; r < 64; r += 16) {
      const int ch = tid & 7;
      const uint16_t* src = z + static_cast<int64_t>(row[r]) * side.ldz;
      cp_async16(at + swz(r, ch), src, r < n);
      cp_async16(at + Z_TILE / 2 + swz(r, ch), src + (wide ? 64 : 0), r < n && wide);
    }
#pragma unroll
    for (int u = tid; u < 64 * MT * 4; u += 128) {
      const int r = u / (MT * 4), j = u % (MT * 4) * 4;
      const bool ok = r < n && j < rank;
      cp_async16(at + Z_TILE + u * 16, side.P + (ok ? static_cast<int64_t>(row[r]) * rank + j : 0), ok);
    }
  };
#pragma unroll
  for (int i = 0; i < STAGES - 1; ++i) {
    if (i < steps) load(i, i);
    cp_async_commit();
  }
  for (int done = 0; done < steps; ++done) {
    cp_async_wait<STAGES - 2>();
    __syncthreads();   // this step has landed for all, and the last one's reads are over
    const uint32_t at = base + (done % STAGES) * STAGE;
#pragma unroll
    for (int u = tid; u < 64 * MT * 4; u += 128) {
      const int r = u / (MT * 4), j = u % (MT * 4) * 4;
      const float4 v = *reinterpret_cast<const float4*>(gen + (done % STAGES) * STAGE + Z_TILE + u * 16);
      __nv_bfloat162 a, b, c, d;
      split_bf16x2(make_float2(v.x, v.y), &a, &c);
      split_bf16x2(make_float2(v.z, v.w), &b, &d);
      *reinterpret_cast<uint2*>(hi + r * P_PITCH + j * 2) =
          make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
      *reinterpret_cast<uint2*>(lo + r * P_PITCH + j * 2) =
          make_uint2(*reinterpret_cast<const uint32_t*>(&c), *reinterpret_cast<const uint32_t*>(&d));
    }
    if (done + STAGES - 1 < steps) load(done + STAGES - 1, (done + STAGES - 1) % STAGES);
    cp_async_commit();
    if (tid < 64) {   // step `done` needs its rows no more
      rows[done & 3][tid] = later;
      later = row_of(done + 5);
    }
    __syncthreads();
    const uint32_t pa = smem_u32(hi), pl = smem_u32(lo);
#pragma unroll
    for (int kk = 0; kk < 4; ++kk) {   // 16 rows t a step
      uint32_t b[2][4];   // columns 32 warp .. + 31
#pragma unroll
      for (int h = 0; h < 2; ++h)
        ldmatrix_x4_trans(b[h], at + (warp >> 1) * (Z_TILE / 2) +
                                    swz(16 * kk + (lane & 15), 4 * (warp & 1) + 2 * h + (lane >> 4)));
      const uint32_t off = (16 * kk + (lane & 7) + ((lane >> 4) << 3)) * P_PITCH + ((lane >> 3) & 1) * 16;
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        uint32_t a[4];
        ldmatrix_x4_trans(a, pa + off + 32 * m);
#pragma unroll
        for (int h = 0; h < 4; ++h) mma_16816(acc[m][h], a, b[h >> 1][2 * (h & 1)], b[h >> 1][2 * (h & 1) + 1]);
        ldmatrix_x4_trans(a, pl + off + 32 * m);
#pragma unroll
        for (int h = 0; h < 4; ++h) mma_16816(acc[m][h], a, b[h >> 1][2 * (h & 1)], b[h >> 1][2 * (h & 1) + 1]);
      }
    }
  }
  cp_async_wait<0>();
  __syncthreads();
  const int g = lane >> 2, q = lane & 3;
  if (slices > 1) {
    // the cluster's sums: CTA c takes the quarters i = 4 m + h with i % slices = c of
    // every thread, from all, adds them in order of the slices and stores them
    float4* part = reinterpret_cast<float4*>(gen);   // [slice][i / slices][thread]
    const int own = MT * 4 / slices;
    cluster_sync();   // no ring is in use any more
#pragma unroll
    for (int i = 0; i < 4 * MT; ++i) {
      const uint32_t to = mapa_shared(smem_u32(part + (slice * own + i / slices) * 128 + tid), i % slices);
      const float* v = acc[i >> 2][i & 3];
      asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(to), "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3])
                   : "memory");
    }
    cluster_sync();
    for (int k = 0; k < own; ++k) {
      const int i = k * slices + slice, m = i >> 2, h = i & 3, c = 32 * warp + 8 * h + 2 * q;
      float4 v = part[k * 128 + tid];
      for (int r = 1; r < slices; ++r) {
        const float4 w = part[(r * own + k) * 128 + tid];
        v.x += w.x;
        v.y += w.y;
        v.z += w.z;
        v.w += w.w;
      }
      if (!wide && warp >= 2) continue;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int j = 16 * m + g + 8 * e;
        if (j >= rank) continue;
        const __nv_bfloat162 x = e ? __floats2bfloat162_rn(v.z, v.w) : __floats2bfloat162_rn(v.x, v.y);
        if (transposed) {
          __nv_bfloat16* to = side.G + (static_cast<int64_t>(id) * side.C + col0 + c) * rank + j;
          to[0] = x.x;
          to[rank] = x.y;
        } else {
          *reinterpret_cast<__nv_bfloat162*>(side.G + (static_cast<int64_t>(id) * rank + j) * side.C + col0 + c) = x;
        }
      }
    }
    return;
  }
  if (transposed) {
    // through shared memory as [128 columns][rank], then rows of `rank` elements
    __nv_bfloat16* st = reinterpret_cast<__nv_bfloat16*>(gen);
    constexpr int PITCH = MT * 16 + 8;
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int h = 0; h < 4; ++h)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          st[(32 * warp + 8 * h + 2 * q + (e & 1)) * PITCH + 16 * m + g + 8 * (e >> 1)] = __float2bfloat16_rn(acc[m][h][e]);
    __syncthreads();
    const int words = rank / 8;
    for (int u = tid; u < (wide ? 128 : 64) * words; u += 128) {
      const int c = u / words, j = (u - c * words) * 8;
      *reinterpret_cast<uint4*>(side.G + (static_cast<int64_t>(id) * side.C + col0 + c) * rank + j) =
          *reinterpret_cast<const uint4*>(st + c * PITCH + j);
    }
  } else {
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int h = 0; h < 4; ++h)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int j = 16 * m + g + 8 * e;
          if (j < rank && (wide || warp < 2)) {
            const __nv_bfloat162 v = __floats2bfloat162_rn(acc[m][h][2 * e], acc[m][h][2 * e + 1]);
            *reinterpret_cast<__nv_bfloat162*>(side.G + (static_cast<int64_t>(id) * rank + j) * side.C + col0 + 32 * warp +
                                               8 * h + 2 * q) = v;
          }
        }
  }
}

// launch_after with a cluster along x.
template <class Kernel, class... Args>
cudaError_t launch_clustered(Kernel kern, dim3 grid, unsigned threads, uint32_t smem, unsigned cluster, cudaStream_t s,
                             Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = cluster;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kern, args...);
}

template <int MT>
cudaError_t grad_mt(const GradSide& da, const GradSide& db, int64_t T, const LoraBatch& b, const int* sorted,
                    const int2* span, int num_sms, cudaStream_t s) {
  static SmemOptIn opt;
  constexpr uint32_t smem = (MT == 8 ? 2 : 3) * (2 * 64 * 128 + 64 * MT * 16 * 4) + 2 * 64 * (MT * 32 + 16) + 128;
  static_assert(128 * (MT * 16 + 8) * 2 <= smem - 128, "the transposed result goes through the ring");
  static_assert(128 * MT * 16 * 4 <= smem - 128, "a cluster's sums go through the ring");
  cudaError_t e = opt.ensure(lora_grad_kernel<MT>, smem);
  if (e != cudaSuccess) return e;
  // A cluster splits an adapter's rows while that leaves room on the GPU and four
  // steps to a CTA (the average adapter's).
  const int64_t blocks = (da.C + 127) / 128 + (db.C + 127) / 128, resident = (MT == 1 ? 3 : MT == 2 ? 2 : 1) * num_sms;
  int slices = 1;
  while (slices < (MT == 1 ? 4 : 8) && blocks * b.count * slices * 2 <= resident && T / 64 >= 8LL * slices * b.count) slices *= 2;
  return launch_clustered(lora_grad_kernel<MT>, dim3(static_cast<unsigned>(blocks * slices), b.count), 128, smem,
                          static_cast<unsigned>(slices), s, da, db, b.rank, sorted, span, slices);
}

}  // namespace

cudaError_t launch_lora_shrink(const void* x, int64_t ldx, int64_t T, int64_t K, const void* A, const void* E, int64_t N,
                               const LoraBatch& b, const LoraPlan& p, bool zeroed, float* V, int num_sms,
                               cudaStream_t s) {
  unsigned int* amax = reinterpret_cast<unsigned int*>(p.amax);
  if (!zeroed) {
    cudaError_t e = launch_zero(amax, 1, s);
    if (e != cudaSuccess) return e;
  }
  static SmemOptIn opt;
  cudaError_t e = opt.ensure(lora_shrink_kernel, kShrinkRing + 1024);
  if (e != cudaSuccess) return e;
  ShrinkParams q = {};
  q.T = static_cast<int>(T);
  q.K = static_cast<int>(K);
  q.count = b.count;
  q.rank = b.rank;
  q.n_pad = (b.rank + 15) / 16 * 16;
  q.S = b.S;
  q.plan_tiles = static_cast<int>((T + 255) / 256);
  q.scale = b.scale;
  q.seg_ptr = b.seg_ptr;
  q.seg_adapter = b.seg_adapter;
  q.plan = PlanOut{p.valid_rows, p.tile_count, p.tile_base, p.tile_direct, E ? p.slab_adapter : nullptr, p.row_adapter};
  q.E = static_cast<const uint16_t*>(E);
  q.elements = N * b.rank;
  q.parts = check_parts(q.elements);
  q.second_max = p.second_max;
  q.amax = amax;
  q.V = V;
  q.after = zeroed;
  const uint32_t stage = kShrinkRows * 128 + q.n_pad * 128;
  q.stages = static_cast<int>(kShrinkRing / stage) < kShrinkMaxStages ? static_cast<int>(kShrinkRing / stage) : kShrinkMaxStages;
  // a cluster splits K while three CTAs for each SM leave room, down to four
  // 64-column steps each
  q.items = static_cast<int>(T / kShrinkRows + b.S);
  q.slices = 1;
  while (q.slices < 8 && static_cast<int64_t>(q.items) * q.slices * 2 <= 3LL * num_sms && K / 64 >= 8 * q.slices) q.slices *= 2;
  const int64_t units = q.plan_tiles + (E ? b.count * q.parts : 0);
  // Rows one by one where that takes less.  Measured (ns): a block of a row
  // takes 3, or what its part of the adapter takes from L2 (6.5 TB/s); an item
  // 6500 and 350 for each 64 columns, as many at a time as fit on the GPU.  512
  // rows of 32 requests, rank 16: 704 columns 5.0 us by rows and 7.4 by items,
  // 8192 columns 24 and 15.
  const int64_t resident = 3LL * num_sms, ctas = static_cast<int64_t>(q.items) * q.slices;
  const int64_t by_item = (6500 + 350 * (K / 64) / q.slices) * (ctas > resident ? ctas : resident) / resident;
  const int64_t by_row = 2000 + T * (b.rank / 8) * (K > 1080 ? K / 360 : 3);
  if (T * (b.rank / 8) < (int64_t(1) << 30) && by_row < by_item) {
    // as many threads as a row has 16-byte pieces, where that is fewer
    const unsigned threads = K >= 8 * kRowThreads ? kRowThreads : K <= 8 * 128 ? 128 : static_cast<unsigned>((K / 8 + 31) / 32 * 32);
    return launch_clustered(lora_shrink_rows_kernel, static_cast<unsigned>(T * (b.rank / 8) + units), threads,
                            (b.count + 31) / 32 * 4, 1, s, static_cast<const uint16_t*>(x), ldx,
                            static_cast<const uint16_t*>(A), q);
  }
  CUtensorMap tmX, tmX32, tmA;
  if (!bf16_map(&tmX, x, T, K, ldx, kShrinkRows, true) || !bf16_map(&tmX32, x, T, K, ldx, 32, true) || !bf16_map(&tmA, A, static_cast<int64_t>(b.count) * b.rank, K, K, q.n_pad, true))
    return cudaErrorInvalidValue;
  return launch_clustered(lora_shrink_kernel, static_cast<unsigned>((q.items + (units + q.slices - 1) / q.slices) * q.slices), kShrinkThreads, q.stages * stage + 1024,
                          static_cast<unsigned>(q.slices), s, tmX, tmX32, tmA, q);
}

cudaError_t launch_lora_transpose(const LoraBatch& b, const void* A, void* a_t, int64_t Cin, const void* B, void* b_t,
                                  int64_t Cout, int64_t T, float* amax, int* sorted, int2* span, cudaStream_t s) {
  transpose_kernel<<<dim3(static_cast<unsigned>(Cin / 64 + Cout / 64 + 1), (b.rank + 31) / 32, b.count), 256, 0, s>>>(
      static_cast<const uint16_t*>(A), static_cast<uint16_t*>(a_t), static_cast<int>(Cin), static_cast<const uint16_t*>(B),
      static_cast<uint16_t*>(b_t), static_cast<int>(Cout), b.rank, amax, b, static_cast<int>(T), sorted, span);
  return cudaGetLastError();
}

cudaError_t launch_lora_grads(const float* U, const void* X, int64_t ldx, int64_t Cin, const float* V, const void* dY,
                              int64_t ldy, int64_t Cout, int64_t T, const LoraBatch& b, const int* sorted, const int2* span,
                              void* dA, void* dB, int num_sms, cudaStream_t s) {
  const GradSide da{U, static_cast<const uint16_t*>(X), ldx, static_cast<int>(Cin), static_cast<__nv_bfloat16*>(dA)};
  const GradSide db{V, static_cast<const uint16_t*>(dY), ldy, static_cast<int>(Cout), static_cast<__nv_bfloat16*>(dB)};
  if (b.rank <= 16) return grad_mt<1>(da, db, T, b, sorted, span, num_sms, s);
  if (b.rank <= 32) return grad_mt<2>(da, db, T, b, sorted, span, num_sms, s);
  if (b.rank <= 64) return grad_mt<4>(da, db, T, b, sorted, span, num_sms, s);
  return grad_mt<8>(da, db, T, b, sorted, span, num_sms, s);
}

}  // namespace nvfp4
