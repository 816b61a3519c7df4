// grads.hip -- the global norm of a list of gradients, and clipping by it.
//
// With g the values of all tensors of the list together:
//   norm   N = sqrt(sum g^2), or the largest |g|
//   factor c = min(1, max_norm / (N + 1e-6)); a NaN stays one
//   out    = g * c, rounded once to g's type
//
// How, on gfx950.  Both are streams over HBM: the norm reads the gradients
// once, the clip reads them again (the factor needs all of them) and writes
// them.  The list is cut into 16 KB units that a fixed grid walks; each
// workgroup leaves one partial result, and every workgroup of the clip sums
// the partials itself, all in the same order, so that the factor costs no
// launch of its own and comes out the same in each and in every run.
//
// Sums: a lane squares and adds the 16 bytes x kGradIters values of a unit in
// fp32 and carries the units' sums in fp64, which costs fp64 work once per
// unit.  Squares that leave fp32's range (|g| above 1.8e19 or all below 1e-9
// or so) are noticed from the unit's sum, and that lane's part is then added
// again in fp64, where no square of an fp32 number overflows or vanishes.
//
// What bounds them: memory.  The norm of a 7B-shaped list (291 tensors, 13.48
// GB of bf16, read once as the counters show) takes 1912-1924 us, 7.0 TB/s,
// where reading two arrays without any arithmetic reaches 6.8-7.3; that of a
// 0.6B-shaped one (310 tensors, 1.19 GB) 176-181 us, 6.7 TB/s, and its clip 398-405
// us for 2.38 GB, 5.9 TB/s, where a bare stream that scales them took 370.  One
// 1M tensor takes 3.0 + 4.0 us, two launches.  (Clipping from the list's end,
// where the norm's last reads might still be cached, gained nothing.  Nor would
// a launch that joins the partial results once for all workgroups of the clip:
// given the total, and so without them, the clip of the 0.6B-shaped list takes
// 397-400 us against 394-397 with them, that of the 7B-shaped one 4873-4899
// against 4740-4764.)
#include <exception>
#include <type_traits>

#include "list.h"

namespace sbd {
namespace {

constexpr int kGradBlock = 256;
constexpr int kGradIters = 4;
constexpr int64_t kGradUnitBytes = int64_t(kGradBlock) * 16 * kGradIters;
constexpr int kGradGrid = 2048;  // 8 workgroups on each of 256 CUs
constexpr int64_t kClipWantGrid = 4096, kClipMaxGrid = int64_t(1) << 22;
// Bytes from which a list passes through: the memory-side cache holds 256 MB.
constexpr int64_t kStreamBytes = int64_t(256) << 20;

struct GradEntry {
  const void* g;
  void* out;
  int64_t numel;
  int64_t first_unit;
  int64_t dtype;  // delta_dtype
};

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint16_t u16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));

// One 16-byte vector of each type as floats, and back.
template <int D>
struct Elem;
template <>
struct Elem<DELTA_BF16> {
  typedef uint16_t bits;
  typedef __bf16 num;
  typedef bf16x8 vec;
};
template <>
struct Elem<DELTA_FP16> {
  typedef uint16_t bits;
  typedef _Float16 num;
  typedef f16x8 vec;
};
template <>
struct Elem<DELTA_FP32> {
  typedef uint32_t bits;
  typedef float num;
  typedef f32x4 vec;
};

template <int D>
constexpr int kElems = 16 / int(sizeof(typename Elem<D>::bits));
template <int D>
constexpr int64_t kUnitElems = kGradUnitBytes / int64_t(sizeof(typename Elem<D>::bits));

// The vector at element i of n, zeros behind the end.  kFull: there is no end
// within this unit, so the unit's loads need no branches between them.
template <int D, bool kFull, bool kStream>
__device__ __forceinline__ typename Elem<D>::vec load_part(const void* g, int64_t i, int64_t n) {
  typedef typename Elem<D>::bits bits;
  constexpr int kN = kElems<D>;
  const auto* p = global_ptr(static_cast<const bits*>(g) + i);
  if (kFull || i + kN <= n) return load_any<kStream, typename Elem<D>::vec>(static_cast<const bits*>(g) + i);
  union {
    bits b[kN];
    typename Elem<D>::vec v;
  } u;
#pragma unroll
  for (int k = 0; k < kN; ++k) u.b[k] = i + k < n ? p[k] : bits(0);
  return u.v;
}

template <int D, bool kFull, bool kStream>
__device__ __forceinline__ void store_part(void* out, int64_t i, int64_t n,
                                           const typename Elem<D>::vec& v) {
  typedef typename Elem<D>::bits bits;
  constexpr int kN = kElems<D>;
  auto* p = global_ptr(static_cast<bits*>(out) + i);
  if (kFull || i + kN <= n) {
    store_any<kStream>(static_cast<bits*>(out) + i, v);
    return;
  }
  union {
    typename Elem<D>::vec v;
    bits b[kN];
  } u;
  u.v = v;
#pragma unroll
  for (int k = 0; k < kN; ++k)
    if (i + k < n) p[k] = u.b[k];
}

// One lane's part of a unit.  kFull: the unit lies inside the tensor.
template <int D, bool kFull, bool kStream>
struct Unit {
  static constexpr int kN = kElems<D>;
  typename Elem<D>::vec v[kGradIters];

  static __device__ __forceinline__ int64_t place(int64_t unit, int k) {
    return unit * kUnitElems<D> + (int64_t(k) * kGradBlock + threadIdx.x) * kN;
  }
  __device__ __forceinline__ void load(const GradEntry& e, int64_t unit) {
#pragma unroll
    for (int k = 0; k < kGradIters; ++k)
      v[k] = load_part<D, kFull, kStream>(e.g, place(unit, k), e.numel);
  }
  __device__ __forceinline__ double squares() const {
    float s[kGradIters];
#pragma unroll
    for (int k = 0; k < kGradIters; ++k) {
      s[k] = 0.0f;
#pragma unroll
      for (int i = 0; i < kN; ++i) {
        const float x = float(v[k][i]);
        s[k] = __builtin_fmaf(x, x, s[k]);
      }
    }
    float sum = 0.0f;
#pragma unroll
    for (int k = 0; k < kGradIters; ++k) sum += s[k];
    // fp32 holds the squares of every value that matters to a sum in this range
    if (sum >= 0x1p-60f && sum <= 0x1p+126f) return double(sum);
    double d = 0.0;
#pragma unroll
    for (int k = 0; k < kGradIters; ++k)
#pragma unroll
      for (int i = 0; i < kN; ++i) {
        const double x = double(float(v[k][i]));
        d = __builtin_fma(x, x, d);
      }
    return d;
  }
  // The largest |g| as the bits of a float without its sign: these order as
  // the numbers do, with infinity and then NaN on top.
  __device__ __forceinline__ uint32_t largest() const {
    uint32_t m = 0;
#pragma unroll
    for (int k = 0; k < kGradIters; ++k)
#pragma unroll
      for (int i = 0; i < kN; ++i) {
        const uint32_t b = __float_as_uint(float(v[k][i])) & 0x7fffffffu;
        m = b > m ? b : m;
      }
    return m;
  }
  // g * c.  The product is an fp32 number before it is rounded to g's type: at
  // most 2^-24 of it is lost there, against the half step of 2^-9 (bf16) or
  // 2^-12 (fp16) that the type itself costs.
  __device__ __forceinline__ void store_times(const GradEntry& e, int64_t unit, float c) {
#pragma unroll
    for (int k = 0; k < kGradIters; ++k) {
#pragma unroll
      for (int i = 0; i < kN; ++i) v[k][i] = static_cast<typename Elem<D>::num>(float(v[k][i]) * c);
      store_part<D, kFull, kStream>(e.out, place(unit, k), e.numel, v[k]);
    }
  }
};

// f(unit in registers, its number) for n units of entry e from `first` on; the
// next unit's loads are issued before f.
template <int D, bool kStream, class F>
__device__ __forceinline__ void for_units(const GradEntry& e, int64_t first, int n, const F& f) {
  const int64_t end = first + n, whole = e.numel / kUnitElems<D>;
  const int64_t full_end = end < whole ? end : whole;
  int64_t u = first;
  if (u < full_end) {
    Unit<D, true, kStream> now, next;
    now.load(e, u);
    for (; u < full_end; ++u) {
      if (u + 1 < full_end) next.load(e, u + 1);
      f(now, u);
      now = next;
    }
  }
  if (u < end) {  // at most one unit ends inside
    Unit<D, false, kStream> last;
    last.load(e, u);
    f(last, u);
  }
}

template <bool kStream, class F>
__device__ __forceinline__ void for_units_of(const GradEntry& e, int64_t first, int n, const F& f) {
  if (e.dtype == DELTA_BF16)
    for_units<DELTA_BF16, kStream>(e, first, n, f);
  else if (e.dtype == DELTA_FP16)
    for_units<DELTA_FP16, kStream>(e, first, n, f);
  else
    for_units<DELTA_FP32, kStream>(e, first, n, f);
}

// What two partial results make together; both are kept as doubles (a NaN
// stays one in either form).
template <bool kInf>
__device__ __forceinline__ double join(double a, double b) {
  if (!kInf) return a + b;
  return a > b || a != a ? a : b;
}

// Over the workgroup's 256 lanes, in a fixed order; valid in every lane.
template <bool kInf>
__device__ __forceinline__ double join_group(double d, double* lds) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) d = join<kInf>(d, __shfl_xor(d, o, 64));
  if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = d;
  __syncthreads();
  double r = lds[0];
#pragma unroll
  for (int w = 1; w < kGradBlock / 64; ++w) r = join<kInf>(r, lds[w]);
  return r;
}

template <bool kInf>
__device__ __forceinline__ double join_partials(const double* partials, int n, double* lds) {
  double d = 0.0;
  for (int i = threadIdx.x; i < n; i += kGradBlock) d = join<kInf>(d, partials[i]);
  return join_group<kInf>(d, lds);
}

template <bool kInf, bool kStream>
__global__ __launch_bounds__(kGradBlock) void grad_norm_kernel(const GradEntry* table,
                                                               GradEntry one, int32_t nparams,
                                                               int64_t units, int span,
                                                               double* partials) {
  __shared__ double lds[kGradBlock / 64];
  double d = 0.0;
  for_each_run(table, one, nparams, units, span, [&](const GradEntry& e, int64_t first, int n) {
    for_units_of<kStream>(e, first, n, [&](const auto& unit, int64_t) {
      if constexpr (kInf)
        d = join<true>(d, double(__uint_as_float(unit.largest())));
      else
        d += unit.squares();
    });
  });
  d = join_group<kInf>(d, lds);
  if (threadIdx.x == 0) partials[blockIdx.x] = d;
}

template <bool kInf>
__device__ __forceinline__ float norm_of(double total) {
  return float(kInf ? total : __builtin_sqrt(total));
}

template <bool kInf>
__global__ __launch_bounds__(kGradBlock) void grad_total_kernel(const double* partials, int n,
                                                                double* total, float* norm) {
  __shared__ double lds[kGradBlock / 64];
  const double d = join_partials<kInf>(partials, n, lds);
  if (threadIdx.x == 0) {
    if (total) *total = d;
    if (norm) *norm = norm_of<kInf>(d);
  }
}

template <bool kInf, bool kStream>
__global__ __launch_bounds__(kGradBlock) void grad_clip_kernel(const GradEntry* table,
                                                               GradEntry one, int32_t nparams,
                                                               int64_t units, int span,
                                                               const double* partials, int n,
                                                               const double* total,
                                                               double max_norm, bool in_place,
                                                               float* norm) {
  __shared__ double lds[kGradBlock / 64];
  const double d = total ? *total : join_partials<kInf>(partials, n, lds);
  const float size = norm_of<kInf>(d);
  const double want = max_norm / (double(size) + 1e-6);
  const float c = want > 1.0 ? 1.0f : float(want);  // a NaN is not above 1
  if (blockIdx.x == 0 && threadIdx.x == 0 && norm) *norm = size;
  // times 1 is what is there already
  if (in_place && c == 1.0f) return;
  for_each_run(table, one, nparams, units, span, [&](const GradEntry& e, int64_t first, int k) {
    for_units_of<kStream>(e, first, k, [&](auto& unit, int64_t u) { unit.store_times(e, u, c); });
  });
}

constexpr size_t kPartialBytes = sizeof(double) * kGradGrid;

size_t grad_ws_bytes(int32_t nparams) {
  return kPartialBytes + sizeof(GradEntry) * (size_t(nparams) + 1);
}

struct GradList {
  std::vector<GradEntry> table;
  int64_t units = 0, bytes = 0;
  bool in_place = true;
};

constexpr int64_t kMaxBytes = int64_t(1) << 61;  // the sum of two stays in range

// Checks the list and lays out its table.
delta_status make_list(const char* fn, int32_t nparams, const void* const* grads,
                       void* const* outs, const int64_t* numels, const int32_t* dtypes,
                       bool writes, bool stored, GradList* list) {
  if (nparams < 0) return fail_with(DELTA_E_INVALID, "%s: nparams=%d < 0", fn, nparams);
  if (nparams > 0 && (grads == nullptr || numels == nullptr || dtypes == nullptr))
    return fail_with(DELTA_E_INVALID, "%s: null parameter array", fn);
  list->table.resize(size_t(nparams) + 1);
  std::vector<Range> ranges;
  int64_t units = 0, bytes = 0;
  for (int32_t p = 0; p < nparams; ++p) {
    const int64_t n = numels[p];
    if (n < 0) return fail_with(DELTA_E_INVALID, "%s: numels[%d]=%lld < 0", fn, p, (long long)n);
    if (dtypes[p] != DELTA_BF16 && dtypes[p] != DELTA_FP16 && dtypes[p] != DELTA_FP32)
      return fail_with(DELTA_E_INVALID, "%s: dtypes[%d]=%d", fn, p, dtypes[p]);
    const int64_t size = dtypes[p] == DELTA_FP32 ? 4 : 2;
    if (n > kMaxBytes / size)
      return fail_with(DELTA_E_RANGE, "%s: numels[%d]=%lld", fn, p, (long long)n);
    void* out = outs ? outs[p] : const_cast<void*>(grads[p]);
    if (n > 0 && (grads[p] == nullptr || (writes && out == nullptr)))
      return fail_with(DELTA_E_INVALID, "%s: null tensor pointer for parameter %d", fn, p);
    const uintptr_t g = reinterpret_cast<uintptr_t>(grads[p]), o = reinterpret_cast<uintptr_t>(out);
    if ((g | (writes ? o : 0)) % uintptr_t(size))
      return fail_with(DELTA_E_INVALID, "%s: parameter %d is not aligned to its elements", fn, p);
    if (out != grads[p]) list->in_place = false;
    list->table[p] = GradEntry{grads[p], out, n, units, dtypes[p]};
    const int64_t per = kGradUnitBytes / size;
    units += (n + per - 1) / per;
    bytes += n * size;
    if (bytes > kMaxBytes)
      return fail_with(DELTA_E_RANGE, "%s: the list holds more than 2^61 bytes", fn);
    if (writes && !stored) {
      ranges.push_back(Range{o, o + uintptr_t(n * size), true});
      if (o != g) ranges.push_back(Range{g, g + uintptr_t(n * size), false});
    }
  }
  list->table[nparams] = GradEntry{nullptr, nullptr, 0, units, 0};
  list->units = units;
  list->bytes = bytes;
  if (ranges_clash(ranges))
    return fail_with(DELTA_E_INVALID, "%s: a tensor that is written overlaps another one", fn);
  return DELTA_OK;
}

// f(kInf, kStream) with both as types.
template <class F>
void by_kind(bool inf, bool stream, const F& f) {
  if (inf)
    stream ? f(std::true_type(), std::true_type()) : f(std::true_type(), std::false_type());
  else
    stream ? f(std::false_type(), std::true_type()) : f(std::false_type(), std::false_type());
}

// One tensor travels as a kernel argument; a longer list has a table.
hipError_t put_table(const GradList& list, int32_t nparams, bool stored, void* ws, hipStream_t s,
                     const GradEntry** d_table) {
  *d_table = nullptr;
  if (nparams == 1) return hipSuccess;
  GradEntry* t = reinterpret_cast<GradEntry*>(static_cast<char*>(ws) + kPartialBytes);
  *d_table = t;
  if (stored) return hipSuccess;
  return store_table(t, list.table.data(), sizeof(GradEntry) * list.table.size(), s);
}

delta_status norm_impl(const char* fn, int32_t nparams, const GradList& list, bool inf,
                       bool stored, void* ws, hipStream_t s, const GradEntry** d_table, int* grid) {
  hipError_t e = put_table(list, nparams, stored, ws, s, d_table);
  if (e != hipSuccess) return hip_result(fn, e);
  const int span = span_for(list.units, kGradGrid, 8);
  *grid = grid_for(list.units, span, kGradGrid);
  double* partials = static_cast<double*>(ws);
  clear_stale_error();
  by_kind(inf, list.bytes >= kStreamBytes, [&](auto i, auto st) {
    grad_norm_kernel<decltype(i)::value, decltype(st)::value><<<*grid, kGradBlock, 0, s>>>(
        *d_table, list.table[0], nparams, list.units, span, partials);
  });
  return hip_result(fn, hipGetLastError());
}

}  // namespace
}  // namespace sbd

extern "C" {

size_t grad_workspace_size(int32_t nparams) {
  return nparams < 0 ? 0 : sbd::grad_ws_bytes(nparams);
}

delta_status grad_list_store(int32_t nparams, const void* const* grad_ptrs, void* const* out_ptrs,
                             const int64_t* numels, const int32_t* dtypes, void* ws,
                             size_t ws_bytes, void* stream) try {
  using namespace sbd;
  const char* fn = "grad_list_store";
  GradList list;
  delta_status st =
      make_list(fn, nparams, grad_ptrs, out_ptrs, numels, dtypes, true, false, &list);
  if (st != DELTA_OK) return st;
  st = check_workspace(fn, ws, ws_bytes, grad_ws_bytes(nparams));
  if (st != DELTA_OK) return st;
  const GradEntry* d_table;
  return hip_result(fn, put_table(list, nparams, false, ws, static_cast<hipStream_t>(stream),
                                  &d_table));
} catch (const std::exception& e) {
  return sbd::fail_with(DELTA_E_INVALID, "grad_list_store: %s", e.what());
}

delta_status grad_norm_many(int32_t nparams, const void* const* grad_ptrs, const int64_t* numels,
                            const int32_t* dtypes, int32_t norm_kind, double* total, float* norm,
                            void* ws, size_t ws_bytes, int32_t table_stored, void* stream) try {
  using namespace sbd;
  const char* fn = "grad_norm_many";
  if (norm_kind != DELTA_NORM_2 && norm_kind != DELTA_NORM_INF)
    return fail_with(DELTA_E_INVALID, "%s: norm_kind=%d", fn, norm_kind);
  if (total == nullptr && norm == nullptr)
    return fail_with(DELTA_E_INVALID, "%s: total and norm are both null", fn);
  GradList list;
  delta_status st = make_list(fn, nparams, grad_ptrs, nullptr, numels, dtypes, false, true, &list);
  if (st != DELTA_OK) return st;
  st = check_workspace(fn, ws, ws_bytes, grad_ws_bytes(nparams));
  if (st != DELTA_OK) return st;
  const bool inf = norm_kind == DELTA_NORM_INF;
  hipStream_t s = static_cast<hipStream_t>(stream);
  const GradEntry* d_table;
  int grid;
  st = norm_impl(fn, nparams, list, inf, table_stored != 0, ws, s, &d_table, &grid);
  if (st != DELTA_OK) return st;
  if (inf)
    grad_total_kernel<true><<<1, kGradBlock, 0, s>>>(static_cast<double*>(ws), grid, total, norm);
  else
    grad_total_kernel<false><<<1, kGradBlock, 0, s>>>(static_cast<double*>(ws), grid, total, norm);
  return hip_result(fn, hipGetLastError());
} catch (const std::exception& e) {
  return sbd::fail_with(DELTA_E_INVALID, "grad_norm_many: %s", e.what());
}

delta_status grad_clip_many(int32_t nparams, const void* const* grad_ptrs, void* const* out_ptrs,
                            const int64_t* numels, const int32_t* dtypes, int32_t norm_kind,
                            const double* total, double max_norm, float* norm, void* ws,
                            size_t ws_bytes, int32_t table_stored, void* stream) try {
  using namespace sbd;
  const char* fn = "grad_clip_many";
  if (norm_kind != DELTA_NORM_2 && norm_kind != DELTA_NORM_INF)
    return fail_with(DELTA_E_INVALID, "%s: norm_kind=%d", fn, norm_kind);
  if (!(max_norm >= 0.0)) return fail_with(DELTA_E_INVALID, "%s: max_norm=%g", fn, max_norm);
  GradList list;
  delta_status st = make_list(fn, nparams, grad_ptrs, out_ptrs, numels, dtypes, true,
                              table_stored != 0, &list);
  if (st != DELTA_OK) return st;
  st = check_workspace(fn, ws, ws_bytes, grad_ws_bytes(nparams));
  if (st != DELTA_OK) return st;
  const bool inf = norm_kind == DELTA_NORM_INF;
  hipStream_t s = static_cast<hipStream_t>(stream);
  const GradEntry* d_table = nullptr;
  int partials = 0;
  if (total == nullptr) {
    st = norm_impl(fn, nparams, list, inf, table_stored != 0, ws, s, &d_table, &partials);
    if (st != DELTA_OK) return st;
  } else {
    const hipError_t e = put_table(list, nparams, table_stored != 0, ws, s, &d_table);
    if (e != hipSuccess) return hip_result(fn, e);
    clear_stale_error();
  }
  const int span = span_for(list.units, kClipWantGrid, 2);
  const int grid = grid_for(list.units, span, kClipMaxGrid);
  by_kind(inf, list.bytes >= kStreamBytes, [&](auto i, auto st2) {
    grad_clip_kernel<decltype(i)::value, decltype(st2)::value><<<grid, kGradBlock, 0, s>>>(
        d_table, list.table[0], nparams, list.units, span, static_cast<double*>(ws), partials, total,
        max_norm, list.in_place, norm);
  });
  return hip_result(fn, hipGetLastError());
} catch (const std::exception& e) {
  return sbd::fail_with(DELTA_E_INVALID, "grad_clip_many: %s", e.what());
}

}  // extern "C"
