// Tokens sorted by expert and back for gfx950 (MI355X): the plan of an expert
// layer's token groups, the copy of tokens into them, the weighted sum of the
// experts' answers, and the gradients of both moves. Formulas: moe_tokens.h.
//
// The sort is a stable counting sort: E + 1 buckets, the last one for dropped
// slots. A wave takes 64 slots at a time; the lanes that hold the same bucket
// find each other with one ballot per bucket bit (the AND over the bits of the
// ballot or its complement), so a lane's place among them is a popcount and
// the lowest one moves the bucket's counter: no atomics, the same plan on
// every run. Up to 16384 slots (and 2048 experts, or no slots) one workgroup does it
// all in one launch: counts per wave, a scan over waves and buckets in LDS,
// placement. Beyond, counts per run of 1024 slots, a scan along the runs of each
// bucket (from 65 runs on; fewer are added up by the next kernel), placement.
//
// The moves are HBM-bound copies. They go token by token, not sorted row by
// row: a token's row is read once and written to its k places, and its k
// answers are read once and summed in registers, so nothing is read k times.

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <mutex>

#include "group_table.h"
#include "moe/moe_tokens.h"
#include "mx_rearrange.h"

namespace {

constexpr int kMaxTopk = 64;
constexpr int kMaxExperts = 4096;
constexpr int64_t kMaxCols = int64_t(1) << 24;
constexpr int64_t kMaxStride = int64_t(1) << 26;
constexpr int kRunSlots = 1024;             // slots per workgroup of the three-launch sort
constexpr int kRunWaves = 4;
constexpr int kMaxWaves = 16;               // of the one-workgroup sort: 16 x 64 slots each at most
constexpr int kSummedRuns = 64;
constexpr int kSortLds = 144 * 1024;        // counters at most: 17 x 2049 or 6 x 4097 words

struct SortParams {
  const void *ids;
  int64_t ld;
  int wide;         // ids are int64
  int topk;
  int slots;
  int experts;
  int32_t *ends, *order, *position;
  int32_t *counts;  // three-launch sort: [bucket][run], then the bucket totals
  int runs;
};

// Bucket of slot i: its expert, or `experts` for a dropped slot.
__device__ __forceinline__ int bucket_of(const SortParams &p, int i) {
  const int t = i / p.topk;
  const int64_t at = int64_t(t) * p.ld + (i - t * p.topk);
  const int64_t id = p.wide ? reinterpret_cast<const int64_t *>(p.ids)[at]
                            : int64_t(reinterpret_cast<const int32_t *>(p.ids)[at]);
  return id >= 0 && id < p.experts ? int(id) : p.experts;
}

// Lanes of the wave that hold the same bucket as this one (idle lanes: none).
__device__ __forceinline__ uint64_t peers(int bucket, bool live, int bits) {
  uint64_t m = __ballot(live);
  for (int b = 0; b < bits; ++b) {
    const bool set = (bucket >> b) & 1;
    const uint64_t v = __ballot(set);
    m &= set ? v : ~v;
  }
  return m;
}

// A wave's share of the slots, from `lo` on, 64 at a time: the buckets in registers, -1 past `hi`. Both passes
// below use them, and all their loads are under way together.
template <int N>
struct Share {
  int bucket[N];
};

template <int N>
__device__ __forceinline__ void load_share(const SortParams &p, int lo, int hi, Share<N> &s) {
  const int lane = threadIdx.x & (kWave - 1);
#pragma unroll
  for (int i = 0; i < N; ++i) s.bucket[i] = lo + i * kWave + lane < hi ? bucket_of(p, lo + i * kWave + lane) : -1;
}

// With PLACE, each slot takes the next row of its bucket from `counter` and is written to the plan; without, only
// counted.
template <bool PLACE, int N>
__device__ __forceinline__ void wave_pass(const SortParams &p, int lo, int hi, const Share<N> &s, int bits,
                                          volatile int *counter) {
  const int lane = threadIdx.x & (kWave - 1);
  const uint64_t below = (uint64_t(1) << lane) - 1;
#pragma unroll
  for (int k = 0; k < N; ++k) {
    if (lo + k * kWave >= hi) break;     // the same for the whole wave
    const int i = lo + k * kWave + lane;
    const int b = s.bucket[k];
    const bool live = b >= 0;
    const uint64_t same = peers(b, live, bits);
    int first = 0;
    if (live) first = counter[b];
    __builtin_amdgcn_wave_barrier();     // every lane has read its counter before the leaders move them
    if (live && (same & below) == 0) counter[b] = first + __popcll(same);
    __builtin_amdgcn_wave_barrier();
    if (PLACE && live) {
      const int row = first + __popcll(same & below);
      const bool dropped = b == p.experts;
      p.position[i] = dropped ? ~row : row;
      p.order[row] = dropped ? ~i : i;
    }
  }
}

// In place over [0, n): the wave's running sums, exclusive, from `carry`.
__device__ __forceinline__ void wave_exclusive_scan(int *v, int n) {
  const int lane = threadIdx.x & (kWave - 1);
  int carry = 0;
  for (int base = 0; base < n; base += kWave) {
    const int x = base + lane < n ? v[base + lane] : 0;
    const int s = wave_inclusive_sum(x) + carry;
    if (base + lane < n) v[base + lane] = s - x;
    carry = __builtin_amdgcn_readlane(s, kWave - 1);
  }
}

__device__ __forceinline__ int bits_for(int buckets) { return 32 - __builtin_clz(unsigned(buckets)); }

// Everything in one workgroup of `waves` waves with up to 64 * N slots each. LDS:
// waves x buckets counters and one total per bucket.
template <int N>
__global__ __launch_bounds__(1024) void sort_one_group(SortParams p) {
  extern __shared__ __align__(16) int sort_lds[];
  const int waves = int(blockDim.x) / kWave;
  const int wave = __builtin_amdgcn_readfirstlane(int(threadIdx.x) / kWave);
  const int buckets = p.experts + 1;
  const int bits = bits_for(buckets);
  int *totals = sort_lds + waves * buckets;
  for (int i = threadIdx.x; i < waves * buckets; i += int(blockDim.x)) sort_lds[i] = 0;
  __syncthreads();
  const int share = ((p.slots + waves - 1) / waves + kWave - 1) / kWave * kWave;   // slots per wave
  const int lo = min(wave * share, p.slots), hi = min(lo + share, p.slots);
  Share<N> mine;
  load_share(p, lo, hi, mine);
  wave_pass<false>(p, lo, hi, mine, bits, sort_lds + wave * buckets);
  __syncthreads();
  for (int b = threadIdx.x; b < buckets; b += int(blockDim.x)) {
    int sum = 0;
    for (int w = 0; w < waves; ++w) {
      const int n = sort_lds[w * buckets + b];
      sort_lds[w * buckets + b] = sum;
      sum += n;
    }
    totals[b] = sum;
  }
  __syncthreads();
  if (wave == 0) wave_exclusive_scan(totals, buckets);
  __syncthreads();
  for (int b = threadIdx.x; b < buckets; b += int(blockDim.x)) {
    const int start = totals[b];
    for (int w = 0; w < waves; ++w) sort_lds[w * buckets + b] += start;
    if (b > 0) p.ends[b - 1] = start;
  }
  __syncthreads();
  wave_pass<true>(p, lo, hi, mine, bits, sort_lds + wave * buckets);
}

// Counts of one run of slots: counts[bucket * runs + run].
__global__ __launch_bounds__(kRunWaves *kWave) void sort_count(SortParams p) {
  extern __shared__ __align__(16) int sort_lds[];
  const int buckets = p.experts + 1;
  for (int b = threadIdx.x; b < buckets; b += int(blockDim.x)) sort_lds[b] = 0;
  __syncthreads();
  const int lo = int(blockIdx.x) * kRunSlots, hi = min(lo + kRunSlots, p.slots);
#pragma unroll
  for (int k = 0; k < kRunSlots / (kRunWaves * kWave); ++k) {
    const int i = lo + k * kRunWaves * kWave + int(threadIdx.x);
    if (i < hi) atomicAdd(&sort_lds[bucket_of(p, i)], 1);
  }
  __syncthreads();
  for (int b = threadIdx.x; b < buckets; b += int(blockDim.x)) p.counts[int64_t(b) * p.runs + blockIdx.x] = sort_lds[b];
}

// One wave per bucket: its counts become the places before each run, its total goes behind them all.
__global__ __launch_bounds__(kWave) void sort_scan(SortParams p) {
  const int lane = threadIdx.x & (kWave - 1);
  int32_t *v = p.counts + int64_t(blockIdx.x) * p.runs;
  int carry = 0;
  for (int base = 0; base < p.runs; base += kWave) {
    const int x = base + lane < p.runs ? v[base + lane] : 0;
    const int s = wave_inclusive_sum(x) + carry;
    if (base + lane < p.runs) v[base + lane] = s - x;
    carry = __builtin_amdgcn_readlane(s, kWave - 1);
  }
  if (lane == 0) p.counts[int64_t(p.experts + 1) * p.runs + blockIdx.x] = carry;
}

// Placement of one run. LDS: a counter for each wave and bucket, the bucket starts. SCANNED: the counts are places
// already (sort_scan); otherwise they are summed here.
template <bool SCANNED>
__global__ __launch_bounds__(kRunWaves *kWave) void sort_place(SortParams p) {
  extern __shared__ __align__(16) int sort_lds[];
  const int buckets = p.experts + 1;
  const int bits = bits_for(buckets);
  const int wave = __builtin_amdgcn_readfirstlane(int(threadIdx.x) / kWave);
  int *starts = sort_lds + kRunWaves * buckets;
  int *before = starts + buckets;      // of this run's bucket
  constexpr int share = kRunSlots / kRunWaves;
  const int run = int(blockIdx.x);
  const int lo = min(run * kRunSlots + wave * share, p.slots), hi = min(lo + share, p.slots);
  Share<share / kWave> mine;
  load_share(p, lo, hi, mine);
  for (int i = threadIdx.x; i < kRunWaves * buckets; i += int(blockDim.x)) sort_lds[i] = 0;
  for (int b = threadIdx.x; b < buckets; b += int(blockDim.x)) {
    const int32_t *v = p.counts + int64_t(b) * p.runs;
    if (SCANNED) {
      starts[b] = p.counts[int64_t(buckets) * p.runs + b];
      before[b] = v[run];
    } else {
      int sum = 0, mid = 0;
#pragma unroll 8
      for (int i = 0; i < p.runs; ++i) {
        if (i == run) mid = sum;
        sum += v[i];
      }
      starts[b] = sum;
      before[b] = mid;
    }
  }
  __syncthreads();
  wave_pass<false>(p, lo, hi, mine, bits, sort_lds + wave * buckets);
  if (wave == 0) wave_exclusive_scan(starts, buckets);
  __syncthreads();
  for (int b = threadIdx.x; b < buckets; b += int(blockDim.x)) {
    int at = starts[b] + before[b];
    for (int w = 0; w < kRunWaves; ++w) {
      const int n = sort_lds[w * buckets + b];
      sort_lds[w * buckets + b] = at;
      at += n;
    }
    if (run == 0 && b > 0) p.ends[b - 1] = starts[b];
  }
  __syncthreads();
  wave_pass<true>(p, lo, hi, mine, bits, sort_lds + wave * buckets);
}

// ------------------------------------------------------------- moves

// 16 bytes of a row: V values of type T, moved with one load or store at the
// type's own alignment (global memory takes dwordx4 accesses at any).
template <class T>
struct Piece {
  static constexpr int V = 16 / int(sizeof(T));
  T v[V];
};

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
template <int ALIGN>
struct Unaligned;
template <>
struct Unaligned<2> {
  typedef u32x4 type __attribute__((aligned(2)));
};
template <>
struct Unaligned<4> {
  typedef u32x4 type __attribute__((aligned(4)));
};

template <class T>
__device__ __forceinline__ Piece<T> load_piece(const T *p, int n) {
  typedef typename Unaligned<sizeof(T)>::type piece_t;
  Piece<T> r;
  if (n >= Piece<T>::V) {
    const u32x4 v = *reinterpret_cast<const piece_t *>(p);
    __builtin_memcpy(&r, &v, 16);
  } else {
#pragma unroll
    for (int i = 0; i < Piece<T>::V; ++i) r.v[i] = i < n ? p[i] : T(0);
  }
  return r;
}

template <class T>
__device__ __forceinline__ void store_piece(T *p, const Piece<T> &r, int n) {
  typedef typename Unaligned<sizeof(T)>::type piece_t;
  if (n >= Piece<T>::V) {
    u32x4 v;
    __builtin_memcpy(&v, &r, 16);
    __builtin_nontemporal_store(v, reinterpret_cast<piece_t *>(p));
  } else {
#pragma unroll
    for (int i = 0; i < Piece<T>::V; ++i)
      if (i < n) p[i] = r.v[i];
  }
}

// 128: seven pieces of 7168 columns divide among them. Measured on 131072 sorted rows of 7168 bf16: the sum 372 us
// (5.7 TB/s; 256 threads 386, 512 384), its gradients 816 us (4.9 TB/s; 64: 855, 256: 828, 512: 895).
constexpr int kMoveThreads = 128;

struct MoveParams {
  const void *src;      // gather: x; combine: y
  void *dst;
  const int32_t *position;
  const float *weights;
  int64_t src_ld, dst_ld;
  int64_t slots;
  int topk;
  int cols;
  int chunks;           // workgroups per token
  // backward of the sum
  const void *dout;
  int64_t dout_ld;
  float *dweights;
};

// A token's positions and weights, slot j in lane j: one load each for all of them, then read lane by lane (as
// scalar loads they are one latency behind another). A lane whose columns lie past the row stays to hold its slot: what
// a lane's register holds once it has left is not defined. load_piece and store_piece touch nothing for it (n <= 0).
struct Slots {
  int pos;
  float weight;
  __device__ __forceinline__ int at(int j) const { return __builtin_amdgcn_readlane(pos, j); }
  __device__ __forceinline__ float weight_at(int j) const {
    return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(weight), j));
  }
};

__device__ __forceinline__ Slots load_slots(const MoveParams &p, int64_t t) {
  const int j = threadIdx.x & (kWave - 1);
  Slots s = {-1, 1.0f};
  if (j < p.topk) {
    s.pos = p.position[t * p.topk + j];
    if (p.weights) s.weight = p.weights[t * p.topk + j];
  }
  return s;
}

template <class T>
__global__ __launch_bounds__(kMoveThreads) void gather_kernel(MoveParams p) {
  const uint32_t t = blockIdx.x / uint32_t(p.chunks);
  const int c = (int(blockIdx.x - t * uint32_t(p.chunks)) * kMoveThreads + int(threadIdx.x)) * Piece<T>::V;
  const int n = p.cols - c;
  const Slots s = load_slots(p, t);
  const Piece<T> v = load_piece(static_cast<const T *>(p.src) + t * p.src_ld + c, n);
  const Piece<T> zero = {};
  for (int j = 0; j < p.topk; ++j) {
    const int pos = s.at(j);
    const int64_t row = pos >= 0 ? pos : ~pos;
    if (row >= p.slots) continue;
    store_piece(static_cast<T *>(p.dst) + row * p.dst_ld + c, pos >= 0 ? v : zero, n);
  }
}

constexpr int kAhead = 8;   // rows of a token's sum that are loaded before the first is used

template <class T>
__global__ __launch_bounds__(kMoveThreads) void combine_kernel(MoveParams p) {
  constexpr int V = Piece<T>::V;
  const uint32_t t = blockIdx.x / uint32_t(p.chunks);
  const int c = (int(blockIdx.x - t * uint32_t(p.chunks)) * kMoveThreads + int(threadIdx.x)) * V;
  const int n = p.cols - c;
  const Slots s = load_slots(p, t);
  float sum[V] = {};
  for (int j0 = 0; j0 < p.topk; j0 += kAhead) {
    Piece<T> v[kAhead];
    bool use[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int pos = j0 + i < p.topk ? s.at(j0 + i) : -1;
      use[i] = pos >= 0 && pos < p.slots;
      if (use[i]) v[i] = load_piece(static_cast<const T *>(p.src) + int64_t(pos) * p.src_ld + c, n);
    }
#pragma unroll
    for (int i = 0; i < kAhead; ++i)
      if (use[i]) {
        const float w = s.weight_at(j0 + i);
#pragma unroll
        for (int k = 0; k < V; ++k) sum[k] = fmaf(w, float(v[i].v[k]), sum[k]);
      }
  }
  Piece<T> r;
#pragma unroll
  for (int k = 0; k < V; ++k) r.v[k] = T(sum[k]);
  store_piece(static_cast<T *>(p.dst) + t * p.dst_ld + c, r, n);
}

__device__ __forceinline__ float wave_sum(float x) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) x += __shfl_xor(x, o, kWave);
  return x;
}

// One workgroup per token: its row of dout is read once for every kAhead slots (it stays in the caches).
template <class T>
__global__ __launch_bounds__(kMoveThreads) void combine_backward_kernel(MoveParams p) {
  constexpr int V = Piece<T>::V;
  constexpr int kWaves = kMoveThreads / kWave;
  __shared__ float partial[kWaves][kAhead];
  const int64_t t = blockIdx.x;
  const int lane = threadIdx.x & (kWave - 1);
  const int wave = int(threadIdx.x) / kWave;
  const T *dout = static_cast<const T *>(p.dout) + t * p.dout_ld;
  const Slots s = load_slots(p, t);
  for (int j0 = 0; j0 < p.topk; j0 += kAhead) {
    float dot[kAhead] = {};
    int pos[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) pos[i] = j0 + i < p.topk ? s.at(j0 + i) : -1;
    for (int c0 = 0; c0 < p.cols; c0 += kMoveThreads * V) {
      const int c = c0 + int(threadIdx.x) * V;
      const int n = p.cols - c;
      const Piece<T> g = load_piece(dout + c, n);
      Piece<T> y[kAhead];
#pragma unroll
      for (int i = 0; i < kAhead; ++i)
        if (pos[i] >= 0 && pos[i] < p.slots)
          y[i] = load_piece(static_cast<const T *>(p.src) + int64_t(pos[i]) * p.src_ld + c, n);
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        if (j0 + i >= p.topk) break;
        const int64_t row = pos[i] >= 0 ? pos[i] : ~pos[i];
        if (row >= p.slots) continue;
        Piece<T> d = {};
        if (pos[i] >= 0) {
          const float w = s.weight_at(j0 + i);
#pragma unroll
          for (int k = 0; k < V; ++k) {
            dot[i] = fmaf(float(g.v[k]), float(y[i].v[k]), dot[i]);
            d.v[k] = T(w * float(g.v[k]));
          }
        }
        store_piece(static_cast<T *>(p.dst) + row * p.dst_ld + c, d, n);
      }
    }
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const float x = wave_sum(dot[i]);
      if (lane == 0) partial[wave][i] = x;
    }
    __syncthreads();
    if (int(threadIdx.x) < kAhead && j0 + int(threadIdx.x) < p.topk) {
      float x = 0.0f;
#pragma unroll
      for (int k = 0; k < kWaves; ++k) x += partial[k][threadIdx.x];
      p.dweights[t * p.topk + j0 + threadIdx.x] = x;
    }
    __syncthreads();
  }
}

int type_bytes(int32_t type) { return type == MOE_F32 ? 4 : 2; }

// Checks shared by the moves; MX_REARRANGE_OK, or the status.
int check_move(int32_t type, int64_t tokens, int32_t topk, int64_t cols) {
  const int64_t lim = (int64_t(1) << 31) - 1 - 4096;
  if (type < MOE_BF16 || type > MOE_F32 || tokens < 0 || cols < 0 || cols > kMaxCols) return MX_REARRANGE_ESHAPE;
  if (topk < 1 || topk > kMaxTopk) return MX_REARRANGE_EGROUPS;
  if (tokens > lim / topk) return MX_REARRANGE_ESHAPE;
  return MX_REARRANGE_OK;
}

bool bad_stride(int64_t ld, int64_t cols) { return ld < cols || ld > kMaxStride; }

int launch(const void *fn, int64_t grid, int threads, size_t lds, void *params, hipStream_t stream) {
  if (grid > max_grid(threads)) return MX_REARRANGE_ESHAPE;
  void *args[] = {params};
  const hipError_t e = hipLaunchKernel(fn, dim3(unsigned(grid)), dim3(unsigned(threads)), args, lds, stream);
  return e == hipSuccess ? MX_REARRANGE_OK : MX_REARRANGE_ELAUNCH;
}

// Launches a kernel of the sort, whose counters may take more LDS than a launch gets unasked.
template <void (*KERNEL)(SortParams)>
int launch_sort(int64_t grid, int threads, size_t lds, SortParams *p, hipStream_t stream) {
  constexpr int kMaxDevices = 64;
  static std::once_flag once[kMaxDevices];
  static bool ready[kMaxDevices];
  const void *fn = reinterpret_cast<const void *>(KERNEL);
  if (lds > 64 * 1024) {
    int dev = 0;
    if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= kMaxDevices) return MX_REARRANGE_ELAUNCH;
    std::call_once(once[dev], [dev, fn] {
      ready[dev] = hipFuncSetAttribute(fn, hipFuncAttributeMaxDynamicSharedMemorySize, kSortLds) == hipSuccess;
    });
    if (!ready[dev]) return MX_REARRANGE_ELAUNCH;
  }
  return launch(fn, grid, threads, lds, p, stream);
}

template <template <class> class PICK>
const void *for_type(int32_t type) {
  return type == MOE_BF16 ? PICK<__bf16>::fn() : type == MOE_F16 ? PICK<_Float16>::fn() : PICK<float>::fn();
}
template <class T>
struct Gather {
  static const void *fn() { return reinterpret_cast<const void *>(&gather_kernel<T>); }
};
template <class T>
struct Combine {
  static const void *fn() { return reinterpret_cast<const void *>(&combine_kernel<T>); }
};
template <class T>
struct CombineBackward {
  static const void *fn() { return reinterpret_cast<const void *>(&combine_backward_kernel<T>); }
};

int chunks_of(int64_t cols, int32_t type) {
  const int64_t per = int64_t(kMoveThreads) * (16 / type_bytes(type));
  return int((cols + per - 1) / per);
}

bool misaligned(const void *p, int32_t type) { return reinterpret_cast<uintptr_t>(p) % type_bytes(type) != 0; }

}  // namespace

extern "C" {

int moe_sort_tokens(const void *expert_ids, int32_t id_bytes, int64_t tokens, int32_t topk, int64_t row_stride,
                    int32_t num_experts, int32_t *group_end_offsets, int32_t *order, int32_t *position,
                    void *workspace, hipStream_t stream) {
  const int64_t lim = (int64_t(1) << 31) - 1 - 4096;
  if (tokens < 0 || (id_bytes != 4 && id_bytes != 8) || row_stride < topk || row_stride > kMaxStride)
    return MX_REARRANGE_ESHAPE;
  if (topk < 1 || topk > kMaxTopk || num_experts < 1 || num_experts > kMaxExperts) return MX_REARRANGE_EGROUPS;
  if (tokens > lim / topk) return MX_REARRANGE_ESHAPE;
  const int64_t slots = tokens * topk;
  const int64_t ws = moe_sort_tokens_workspace_bytes(tokens, topk, num_experts);
  if (group_end_offsets == nullptr || (ws > 0 && workspace == nullptr) ||
      (slots > 0 && (expert_ids == nullptr || order == nullptr || position == nullptr)))
    return MX_REARRANGE_ENULL;
  if (reinterpret_cast<uintptr_t>(expert_ids) % unsigned(id_bytes) || reinterpret_cast<uintptr_t>(workspace) % 4)
    return MX_REARRANGE_EALIGN;
  SortParams p = {};
  p.ids = expert_ids;
  p.ld = row_stride;
  p.wide = id_bytes == 8;
  p.topk = topk;
  p.slots = int(slots);
  p.experts = num_experts;
  p.ends = group_end_offsets;
  p.order = order;
  p.position = position;
  const int buckets = num_experts + 1;
  if (ws == 0) {
    int waves = int((slots + kWave - 1) / kWave);     // as many as have 64 slots to work on
    waves = waves < 1 ? 1 : waves > kMaxWaves ? kMaxWaves : waves;
    const int64_t each = (slots + waves - 1) / waves;
    const size_t lds = size_t(waves + 1) * buckets * 4;
    if (each <= kWave) return launch_sort<sort_one_group<1>>(1, waves * kWave, lds, &p, stream);
    if (each <= 4 * kWave) return launch_sort<sort_one_group<4>>(1, waves * kWave, lds, &p, stream);
    return launch_sort<sort_one_group<16>>(1, waves * kWave, lds, &p, stream);
  }
  p.counts = static_cast<int32_t *>(workspace);
  p.runs = int((slots + kRunSlots - 1) / kRunSlots);
  // few runs: every workgroup of the last kernel adds up the earlier runs' counts itself
  const bool scanned = p.runs > kSummedRuns;
  int rc = launch_sort<sort_count>(p.runs, kRunWaves * kWave, size_t(buckets) * 4, &p, stream);
  if (rc == MX_REARRANGE_OK && scanned) rc = launch_sort<sort_scan>(buckets, kWave, 0, &p, stream);
  if (rc == MX_REARRANGE_OK) {
    const size_t lds = size_t(kRunWaves + 2) * buckets * 4;
    rc = scanned ? launch_sort<sort_place<true>>(p.runs, kRunWaves * kWave, lds, &p, stream)
                 : launch_sort<sort_place<false>>(p.runs, kRunWaves * kWave, lds, &p, stream);
  }
  return rc;
}

int moe_gather_tokens(const void *x, int32_t type, int64_t tokens, int32_t topk, int64_t cols, int64_t row_stride,
                      const int32_t *position, void *out, int64_t out_stride, hipStream_t stream) {
  const int rc = check_move(type, tokens, topk, cols);
  if (rc != MX_REARRANGE_OK) return rc;
  if (bad_stride(row_stride, cols) || bad_stride(out_stride, cols)) return MX_REARRANGE_ESHAPE;
  if (tokens * cols == 0) return MX_REARRANGE_OK;   // nothing to write
  if (x == nullptr || position == nullptr || out == nullptr) return MX_REARRANGE_ENULL;
  if (misaligned(x, type) || misaligned(out, type)) return MX_REARRANGE_EALIGN;
  MoveParams p = {};
  p.src = x;
  p.dst = out;
  p.position = position;
  p.src_ld = row_stride;
  p.dst_ld = out_stride;
  p.slots = tokens * topk;
  p.topk = topk;
  p.cols = int(cols);
  p.chunks = chunks_of(cols, type);
  return launch(for_type<Gather>(type), tokens * p.chunks, kMoveThreads, 0, &p, stream);
}

int moe_combine_tokens(const void *y, int32_t type, int64_t tokens, int32_t topk, int64_t cols, int64_t row_stride,
                       const int32_t *position, const float *weights, void *out, int64_t out_stride,
                       hipStream_t stream) {
  const int rc = check_move(type, tokens, topk, cols);
  if (rc != MX_REARRANGE_OK) return rc;
  if (bad_stride(row_stride, cols) || bad_stride(out_stride, cols)) return MX_REARRANGE_ESHAPE;
  if (tokens * cols == 0) return MX_REARRANGE_OK;   // nothing to write
  if (y == nullptr || position == nullptr || out == nullptr) return MX_REARRANGE_ENULL;
  if (misaligned(y, type) || misaligned(out, type)) return MX_REARRANGE_EALIGN;
  MoveParams p = {};
  p.src = y;
  p.dst = out;
  p.position = position;
  p.weights = weights;
  p.src_ld = row_stride;
  p.dst_ld = out_stride;
  p.slots = tokens * topk;
  p.topk = topk;
  p.cols = int(cols);
  p.chunks = chunks_of(cols, type);
  return launch(for_type<Combine>(type), tokens * p.chunks, kMoveThreads, 0, &p, stream);
}

int moe_combine_tokens_backward(const void *dout, int32_t type, int64_t tokens, int32_t topk, int64_t cols,
                                int64_t dout_stride, const void *y, int64_t row_stride, const int32_t *position,
                                const float *weights, void *dy, int64_t dy_stride, float *dweights,
                                hipStream_t stream) {
  const int rc = check_move(type, tokens, topk, cols);
  if (rc != MX_REARRANGE_OK) return rc;
  if (bad_stride(row_stride, cols) || bad_stride(dout_stride, cols) || bad_stride(dy_stride, cols))
    return MX_REARRANGE_ESHAPE;
  if (tokens == 0) return MX_REARRANGE_OK;   // nothing to write
  if (position == nullptr || weights == nullptr || dweights == nullptr ||
      (cols > 0 && (dout == nullptr || y == nullptr || dy == nullptr)))
    return MX_REARRANGE_ENULL;
  if (misaligned(dout, type) || misaligned(y, type) || misaligned(dy, type)) return MX_REARRANGE_EALIGN;
  MoveParams p = {};
  p.src = y;
  p.dst = dy;
  p.position = position;
  p.weights = weights;
  p.src_ld = row_stride;
  p.dst_ld = dy_stride;
  p.slots = tokens * topk;
  p.topk = topk;
  p.cols = int(cols);
  p.dout = dout;
  p.dout_ld = dout_stride;
  p.dweights = dweights;
  return launch(for_type<CombineBackward>(type), tokens, kMoveThreads, 0, &p, stream);
}

}  // extern "C"
