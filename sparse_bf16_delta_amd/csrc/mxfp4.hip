// mxfp4.hip -- the sampler's snapshots as MXFP4: quantising a parameter list,
// its values back, and applying a delta to snapshots and replica together.
//
// The sampler keeps a bf16 snapshot that deltas are applied to (apply.hip) and
// serves from a 4-bit replica of it.  mxfp4.h has the arithmetic of a block.
//
// How, on gfx950.  Quantising and the way back are streams: four neighbouring
// lanes share a block, each with one 16-byte load of 8 bf16 values, so that a
// wave reads 1 KB and writes 256 bytes of elements without gaps; the block's
// largest value is joined across the four lanes by two lane permutations.
//
// A delta is applied and the replica brought up to date in one pass over its
// entries: idx ascends, so the first entry of each touched group of four
// blocks stands for it; sixteen lanes read the group's 256 bytes, its entries
// are put into them in LDS, and the lanes write the touched blocks back and
// quantise the group.  A group belongs to one first entry, so no two workgroups
// meet.  Groups and not blocks, because 64 bytes of codes are written whole
// then: memory reads what a smaller store leaves of them.  Large dense deltas
// touch nearly every block: apply.hip's kernels and a stream over the list do
// it then.
//
// What bounds them, and what they reach.  Quantising 596,049,920 bf16 values
// (310 tensors) takes 242-249 us, the way back 253-263: 1.51 GB each, moved
// once as the counters show, at 6.0-6.2 and 5.8-6.0 TB/s, where bare streams
// of the same bytes took 223 and 236 us.  One 1024 x 1024 tensor takes 2.9-3.1
// us each way, which is a launch.  fp16 goes as bf16 does; fp32 quantises at 5.2
// TB/s and comes back at 2.5 (36 tensors of 4096 x 4096, 531 and 1077 us; bf16
// 247 and 284).  Rows that are no multiple of 32, bf16: 36 tensors of 4096 x 4097
// 294 us and 323 back, 5.2 and 4.7 TB/s, without the next loads in flight and with
// a division for every block.  A delta of 7.2M entries (1.18 %) into 607M
// values takes 382-408 us: 0.77 GB read and 0.58 GB written at 3.4 TB/s, because
// single blocks of 64 bytes are read and written back; without the stores of
// the codes it took 312 us, without those of the snapshot 283.  The same delta
// by apply.hip alone takes 274 us, and another pass over the touched blocks
// took 347 more.
#include <exception>
#include <type_traits>

#include "mxfp4.h"

namespace sbd {
namespace {

constexpr int kMxGroup = 256;  // lanes of a workgroup
constexpr int kMxIters = 2;
constexpr int kMxUnit = kMxGroup / 4 * kMxIters;  // blocks: 8 KB of bf16 values
constexpr int64_t kMxWantGrid = 4096, kMxMaxGrid = int64_t(1) << 22;

struct MxEntry {
  void* x;
  uint8_t* codes;
  uint8_t* scales;
  int64_t first_unit;
  uint32_t rows, cols, row_blocks, dtype;
};

// Where lane `q` of block `b` finds its 8 values, and how many there are.
struct Place {
  int64_t at;
  int valid;
};
__device__ __forceinline__ Place place_of(const MxEntry& e, uint32_t b, uint32_t q) {
  if ((e.cols & 31u) == 0) return Place{int64_t(b) * kMxBlock + q * 8, 8};
  const uint32_t row = b / e.row_blocks;
  const int64_t col = int64_t(b - row * e.row_blocks) * kMxBlock + q * 8;
  const int64_t left = int64_t(e.cols) - col;
  return Place{int64_t(row) * e.cols + col, int(left < 0 ? 0 : left < 8 ? left : 8)};
}

template <int D, bool kStream>
__device__ __forceinline__ void write_block_part(const MxEntry& e, const Eight<D>& v, uint32_t b,
                                                 uint32_t q) {
  const uint32_t byte = scale_byte(Eight<D>::exponent(largest_of_quad(v.largest())));
  const uint32_t codes = byte == 255u ? 0u : v.encode(scale_operand(byte));
  store_any<kStream>(e.codes + int64_t(b) * kMxBlockBytes + q * 4, codes);
  if (q == 0) global_ptr(e.scales)[b] = uint8_t(byte);  // the caches gather single bytes
}

// One unit's values in registers: this lane's 8 of kMxIters blocks, for units
// of whole blocks in memory order.
template <int D, bool kStream>
struct ValueUnit {
  Eight<D> v[kMxIters];
  __device__ __forceinline__ void load(const MxEntry& e, int64_t b, uint32_t q) {
#pragma unroll
    for (int k = 0; k < kMxIters; ++k)
      v[k].template load<kStream>(static_cast<const char*>(e.x) +
                                  ((b + k * (kMxGroup / 4)) * kMxBlock + q * 8) * Eight<D>::kSize);
  }
  __device__ __forceinline__ void finish(const MxEntry& e, int64_t b, uint32_t q) const {
#pragma unroll
    for (int k = 0; k < kMxIters; ++k)
      write_block_part<D, kStream>(e, v[k], uint32_t(b) + k * (kMxGroup / 4), q);
  }
};

// The same for the way back.
template <int D, bool kStream>
struct CodeUnit {
  uint32_t codes[kMxIters];
  uint8_t byte[kMxIters];
  __device__ __forceinline__ void load(const MxEntry& e, int64_t b, uint32_t q) {
#pragma unroll
    for (int k = 0; k < kMxIters; ++k) {
      const int64_t at = b + k * (kMxGroup / 4);
      codes[k] = load_any<kStream, uint32_t>(e.codes + at * kMxBlockBytes + q * 4);
      byte[k] = global_ptr(e.scales)[at];
    }
  }
  __device__ __forceinline__ void finish(const MxEntry& e, int64_t b, uint32_t q) const {
#pragma unroll
    for (int k = 0; k < kMxIters; ++k) {
      const int64_t at = b + k * (kMxGroup / 4);
      Eight<D> v;
      v.decode(codes[k], scale_operand(byte[k]));
      store_any<kStream>(static_cast<char*>(e.x) + (at * kMxBlock + q * 8) * Eight<D>::kSize,
                         v.raw);
    }
  }
};

// n units of entry e from unit `first` on.
template <bool kBack, int D, bool kStream>
__device__ __forceinline__ void do_run(const MxEntry& e, int64_t first, int n) {
  const uint32_t q = threadIdx.x & 3u, mine = threadIdx.x >> 2;
  const uint32_t blocks = e.rows * e.row_blocks;
  // whole units of whole blocks
  const int64_t whole = (e.cols & 31u) == 0 ? blocks / kMxUnit : 0;
  const int64_t end = first + n, plain_end = end < whole ? end : whole;
  int64_t u = first;
  if (u < plain_end) {
    typedef std::conditional_t<kBack, CodeUnit<D, kStream>, ValueUnit<D, kStream>> Unit;
    Unit now, next;
    now.load(e, u * kMxUnit + mine, q);
    for (; u < plain_end; ++u) {
      if (u + 1 < plain_end) next.load(e, (u + 1) * kMxUnit + mine, q);
      now.finish(e, u * kMxUnit + mine, q);
      now = next;
    }
  }
  for (; u < end; ++u) {
    const uint32_t b0 = uint32_t(u) * kMxUnit;
    // four neighbouring lanes share b, so they leave together
    for (uint32_t b = b0 + mine; b < b0 + kMxUnit && b < blocks; b += kMxGroup / 4) {
      const Place at = place_of(e, b, q);
      char* x = static_cast<char*>(e.x) + at.at * Eight<D>::kSize;
      Eight<D> v;
      if (kBack) {
        v.decode(load_any<uint32_t>(e.codes + int64_t(b) * kMxBlockBytes + q * 4),
                 scale_operand(global_ptr(e.scales)[b]));
        store_valid<D>(v, x, at.valid);
      } else {
        load_valid<D>(v, x, at.valid);
        write_block_part<D, kStream>(e, v, b, q);
      }
    }
  }
}

template <bool kBack, bool kStream>
__global__ __launch_bounds__(kMxGroup) void mx_list_kernel(const MxEntry* table, MxEntry one,
                                                           int32_t nparams, int64_t units,
                                                           int span) {
  for_each_run(table, one, nparams, units, span, [](const MxEntry& e, int64_t first, int n) {
    if (e.dtype == DELTA_BF16)
      do_run<kBack, DELTA_BF16, kStream>(e, first, n);
    else if (e.dtype == DELTA_FP16)
      do_run<kBack, DELTA_FP16, kStream>(e, first, n);
    else
      do_run<kBack, DELTA_FP32, kStream>(e, first, n);
  });
}

// Where element i of a tensor lies: its block and its place in it; block -1 for
// an index outside the tensor.
struct Spot {
  int64_t block;
  uint32_t elem;
};
__device__ __forceinline__ Spot spot_of(const MxEntry& e, int32_t i) {
  if (i < 0 || int64_t(i) >= int64_t(e.rows) * e.cols) return Spot{-1, 0};
  if ((e.cols & 31u) == 0) return Spot{int64_t(uint32_t(i) >> 5), uint32_t(i) & 31u};
  const uint32_t row = uint32_t(i) / e.cols, col = uint32_t(i) - row * e.cols;
  return Spot{int64_t(row) * e.row_blocks + (col >> 5), col & 31u};
}

// A workgroup's step: kTile delta entries, and the groups of four blocks (128
// values, 64 bytes of codes) whose first entry is among them, 64 groups at a
// time in LDS.
constexpr int kGroupBlocks = 4;
constexpr int kRound = 64;
// Touched blocks of a group up to which only they are read and written: with
// more, whole groups cost less than stores with gaps.  us for 0 / 1 / 2 / 4 of
// them, 607M values, at 0.3 % of entries 166 / 129 / 129 / 133, at 1.2 % 378 /
// 364 / 371 / 381, at 3 % 514 / 516 / 531 / 547.
constexpr int kBlocksAlone = 1;

template <int kTile>
struct ApplyShared {
  int32_t span[2];  // the parameters of the tile's first and last entry
  uint32_t count[kTile / 64];
  uint32_t group[kTile];
  uint32_t touched[kTile];  // per group: which of its blocks have an entry
  int32_t param[kTile];
  __attribute__((aligned(16))) uint16_t data[kRound * kGroupBlocks * kMxBlock];
};

// What a step's groups come from: entries start .. start + n of the delta;
// entries from `total` on do not exist.
struct ApplyStep {
  const int32_t* idx;
  const uint16_t* val;
  const int64_t* offsets;
  int64_t start, total;
  int n;
  int32_t p_first, p_last;
};

// One step.  kApply: the delta's values are written into the snapshots here;
// else they are there already.  kOne: all its entries belong to e.
template <bool kApply, bool kOne, int kTile>
__device__ __forceinline__ void apply_step(ApplyShared<kTile>& sh, const ApplyStep& st,
                                           const MxEntry* __restrict__ table, const MxEntry& e) {
  typedef Eight<DELTA_BF16> Bf16;
  constexpr int kPer = kTile / kMxGroup;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;

  for (int i = threadIdx.x; i < kTile; i += kMxGroup) sh.touched[i] = 0;
  // Each lane's entries, and which of them is the first of its group: idx
  // ascends, so the entries of a group are neighbours and the first one stands
  // for it.
  int64_t group[kPer];
  uint32_t elem[kPer], value[kPer], before[kPer];  // before: firsts up to the entry, in its wave
  int32_t param[kPer];
  bool first[kPer];
#pragma unroll
  for (int k = 0; k < kPer; ++k) {
    const int i = k * kMxGroup + threadIdx.x;
    const int64_t j = st.start + i;
    group[k] = -1;
    first[k] = false;
    param[k] = st.p_first;
    if (i < st.n) {
      int32_t p = st.p_first;
      MxEntry mine = e;
      if (!kOne) {
        int32_t hi = st.p_last + 1;
        while (hi - p > 1) {
          const int32_t mid = p + (hi - p) / 2;
          if (st.offsets[mid] <= j)
            p = mid;
          else
            hi = mid;
        }
        mine = table[p];
        param[k] = p;
      }
      const Spot at = spot_of(mine, st.idx[j]);
      if (kApply) value[k] = st.val[j];
      if (at.block >= 0) {
        group[k] = at.block / kGroupBlocks;
        elem[k] = uint32_t(at.block % kGroupBlocks) * kMxBlock + at.elem;
        first[k] = true;
        // what lies in front of offsets[0] is parameter 0's
        if (j > 0 && (j > st.offsets[p] || p == 0)) {
          const Spot last = spot_of(mine, st.idx[j - 1]);
          first[k] = last.block < 0 || last.block / kGroupBlocks != group[k];
        }
      }
    }
    const uint64_t mask = __ballot(first[k]);
    before[k] = __popcll(mask & (~uint64_t(0) >> (63 - lane)));
    if (lane == 0) sh.count[k * (kMxGroup / 64) + wave] = __popcll(mask);
  }
  __syncthreads();
  uint32_t groups = 0;
  int32_t slot[kPer];
#pragma unroll
  for (int k = 0; k < kPer; ++k)
#pragma unroll
    for (int w = 0; w < kMxGroup / 64; ++w) {
      // an entry before the step's first group belongs to the step before
      if (w == wave) slot[k] = int32_t(groups + before[k]) - 1;
      groups += sh.count[k * (kMxGroup / 64) + w];
    }
#pragma unroll
  for (int k = 0; k < kPer; ++k) {
    if (group[k] < 0) slot[k] = -1;
    if (first[k]) {
      sh.group[slot[k]] = uint32_t(group[k]);
      if (!kOne) sh.param[slot[k]] = param[k];
    }
    if (slot[k] >= 0) atomicOr(&sh.touched[slot[k]], 1u << (elem[k] / kMxBlock));
  }
  __syncthreads();
  // the last group's entries behind the step
  uint32_t more_elem = 0, more_value = 0;
  bool more = false;
  if (groups > 0 && threadIdx.x < kGroupBlocks * kMxBlock) {
    const int32_t p = kOne ? st.p_first : sh.param[groups - 1];
    const MxEntry mine = kOne ? e : table[p];
    const int64_t stop = st.offsets[p + 1] < st.total ? st.offsets[p + 1] : st.total;
    const int64_t j = st.start + st.n + threadIdx.x;
    if (j < stop) {
      const Spot at = spot_of(mine, st.idx[j]);
      if (at.block >= 0 && at.block / kGroupBlocks == int64_t(sh.group[groups - 1])) {
        more = true;
        more_elem = uint32_t(at.block % kGroupBlocks) * kMxBlock + at.elem;
        if (kApply) more_value = st.val[j];
        atomicOr(&sh.touched[groups - 1], 1u << (more_elem / kMxBlock));
      }
    }
  }
  __syncthreads();

  const uint32_t sub = threadIdx.x & 15u, q = sub & 3u;
  constexpr int kLoads = kRound * 16 / kMxGroup;  // 16 lanes a group
  // A group with one touched block is that block alone; else all of it.
  auto used = [&](uint32_t s) {
    const uint32_t t = sh.touched[s];
    return __popc(t) > kBlocksAlone || (t >> (sub / 4) & 1u);
  };
  for (uint32_t r0 = 0; r0 < groups; r0 += kRound) {
    Bf16 v[kLoads];
#pragma unroll
    for (int g = 0; g < kLoads; ++g) {
      const uint32_t s = r0 + g * (kMxGroup / 16) + threadIdx.x / 16;
      v[g].raw = u32x4{0u, 0u, 0u, 0u};
      if (s >= groups || !used(s)) continue;
      const MxEntry mine = kOne ? e : table[sh.param[s]];
      const uint32_t b = sh.group[s] * kGroupBlocks + sub / 4;
      if (b >= mine.rows * mine.row_blocks) continue;
      const Place at = place_of(mine, b, q);
      load_valid<DELTA_BF16>(v[g], static_cast<const uint16_t*>(mine.x) + at.at, at.valid);
    }
    if (kApply) {
      // the round's values through LDS, where every entry puts its own
#pragma unroll
      for (int g = 0; g < kLoads; ++g)
        *reinterpret_cast<u32x4*>(sh.data + (g * kMxGroup + threadIdx.x) * 8) = v[g].raw;
      __syncthreads();
#pragma unroll
      for (int k = 0; k < kPer; ++k)
        if (slot[k] >= int32_t(r0) && slot[k] < int32_t(r0) + kRound)
          sh.data[(slot[k] - int32_t(r0)) * (kGroupBlocks * kMxBlock) + elem[k]] =
              uint16_t(value[k]);
      if (more && groups - r0 <= kRound)
        sh.data[(groups - 1 - r0) * (kGroupBlocks * kMxBlock) + more_elem] = uint16_t(more_value);
      __syncthreads();
    }
#pragma unroll
    for (int g = 0; g < kLoads; ++g) {
      const uint32_t s = r0 + g * (kMxGroup / 16) + threadIdx.x / 16;
      if (s >= groups || !used(s)) continue;
      const MxEntry mine = kOne ? e : table[sh.param[s]];
      const uint32_t b = sh.group[s] * kGroupBlocks + sub / 4;
      if (b >= mine.rows * mine.row_blocks) continue;  // four lanes leave together
      if (kApply) {
        v[g].raw = *reinterpret_cast<const u32x4*>(sh.data + (g * kMxGroup + threadIdx.x) * 8);
        if (sh.touched[s] >> (sub / 4) & 1u) {
          const Place at = place_of(mine, b, q);
          store_valid<DELTA_BF16>(v[g], static_cast<uint16_t*>(mine.x) + at.at, at.valid);
        }
      }
      write_block_part<DELTA_BF16, false>(mine, v[g], b, q);
    }
    if (kApply) __syncthreads();
  }
}

template <bool kApply, int kTile>
__global__ __launch_bounds__(kMxGroup) void mx_apply_kernel(
    const MxEntry* __restrict__ table, MxEntry one, int32_t nparams,
    const int32_t* __restrict__ idx, const uint16_t* __restrict__ val,
    const int64_t* __restrict__ offsets, int64_t max_nnz) {
  __shared__ ApplyShared<kTile> sh;
  // no entry outside [0, max_nnz) is read
  int64_t total = offsets[nparams];
  total = total < max_nnz ? total : max_nnz;
  for (int64_t start = int64_t(blockIdx.x) * kTile; start < total;
       start += int64_t(gridDim.x) * kTile) {
    const int64_t end = start + kTile < total ? start + kTile : total;
    ApplyStep st{idx, val, offsets, start, total, int(end - start), 0, 0};
    if (table) {
      if (threadIdx.x < 64) {
        const int32_t lo = find_param_wave0(offsets, nparams, start);
        const int32_t hi = find_param_wave0(offsets, nparams, end - 1);
        if (threadIdx.x == 0) {
          sh.span[0] = lo;
          sh.span[1] = hi;
        }
      }
      __syncthreads();
      st.p_first = __builtin_amdgcn_readfirstlane(sh.span[0]);
      st.p_last = __builtin_amdgcn_readfirstlane(sh.span[1]);
    }
    // a step within one tensor, by far the most common, needs no searches
    MxEntry e = one;
    if (table) e = table[st.p_first];
    if (st.p_first == st.p_last)
      apply_step<kApply, true, kTile>(sh, st, table, e);
    else
      apply_step<kApply, false, kTile>(sh, st, table, e);
    __syncthreads();
  }
}

struct MxList {
  std::vector<MxEntry> table;
  int64_t units = 0, elems = 0;
};

constexpr int64_t kMxMaxElems = 2147483647LL;  // as everywhere: int32 positions

// The workspace: this file's table, then that of apply.hip for the same list.
size_t mx_table_bytes(int32_t nparams) {
  return (sizeof(MxEntry) * (size_t(nparams) + 1) + 255) & ~size_t(255);
}
size_t mx_ws_bytes(int32_t nparams) {
  return mx_table_bytes(nparams) + sizeof(SnapParam) * size_t(nparams);
}

// Checks the list and lays out its table.  dtypes null: all bf16.  writes_*:
// what the call writes.
delta_status make_list(const char* fn, int32_t nparams, void* const* xs, const int32_t* dtypes,
                       const int64_t* rows, const int64_t* cols, uint8_t* const* codes,
                       uint8_t* const* scales, bool writes_x, bool writes_codes, bool stored,
                       MxList* list) {
  if (nparams < 0) return fail_with(DELTA_E_INVALID, "%s: nparams=%d < 0", fn, nparams);
  if (nparams > 0 && (xs == nullptr || rows == nullptr || cols == nullptr || codes == nullptr ||
                      scales == nullptr))
    return fail_with(DELTA_E_INVALID, "%s: null parameter array", fn);
  list->table.resize(size_t(nparams) + 1);
  std::vector<Range> ranges;
  int64_t units = 0;
  for (int32_t p = 0; p < nparams; ++p) {
    const int64_t r = rows[p], c = cols[p];
    if (r < 0 || c < 0)
      return fail_with(DELTA_E_INVALID, "%s: parameter %d has shape %lld x %lld", fn, p,
                       (long long)r, (long long)c);
    if (r > kMxMaxElems || c > kMxMaxElems || (c > 0 && r > kMxMaxElems / c))
      return fail_with(DELTA_E_RANGE, "%s: parameter %d (%lld x %lld) exceeds the int32 index range",
                       fn, p, (long long)r, (long long)c);
    const int32_t dtype = dtypes ? dtypes[p] : int32_t(DELTA_BF16);
    if (dtype != DELTA_BF16 && dtype != DELTA_FP16 && dtype != DELTA_FP32)
      return fail_with(DELTA_E_INVALID, "%s: dtypes[%d]=%d", fn, p, dtype);
    const int64_t row_blocks = (c + kMxBlock - 1) / kMxBlock, blocks = r * row_blocks;
    if (blocks > 0 && (xs[p] == nullptr || codes[p] == nullptr || scales[p] == nullptr))
      return fail_with(DELTA_E_INVALID, "%s: null tensor pointer for parameter %d", fn, p);
    const int64_t size = dtype == DELTA_FP32 ? 4 : 2;
    const uintptr_t x = reinterpret_cast<uintptr_t>(xs[p]);
    const uintptr_t cd = reinterpret_cast<uintptr_t>(codes[p]);
    const uintptr_t sc = reinterpret_cast<uintptr_t>(scales[p]);
    if (x % uintptr_t(size))
      return fail_with(DELTA_E_INVALID, "%s: parameter %d is not aligned to its elements", fn, p);
    list->table[p] = MxEntry{xs[p],       codes[p],    scales[p],           units,
                             uint32_t(r), uint32_t(c), uint32_t(row_blocks), uint32_t(dtype)};
    units += (blocks + kMxUnit - 1) / kMxUnit;
    list->elems += r * c;
    if (!stored) {
      ranges.push_back(Range{x, x + uintptr_t(r * c * size), writes_x});
      ranges.push_back(Range{cd, cd + uintptr_t(blocks * kMxBlockBytes), writes_codes});
      ranges.push_back(Range{sc, sc + uintptr_t(blocks), writes_codes});
    }
  }
  list->table[nparams] = MxEntry{nullptr, nullptr, nullptr, units, 0, 0, 0, 0};
  list->units = units;
  if (ranges_clash(ranges))
    return fail_with(DELTA_E_INVALID, "%s: a tensor that is written overlaps another one", fn);
  return DELTA_OK;
}

// One tensor travels as a kernel argument; a longer list has a table.
hipError_t put_table(const MxList& list, int32_t nparams, bool stored, void* ws, hipStream_t s,
                     const MxEntry** d_table) {
  *d_table = nullptr;
  if (nparams == 1) return hipSuccess;
  *d_table = static_cast<MxEntry*>(ws);
  if (stored) return hipSuccess;
  return store_table(ws, list.table.data(), sizeof(MxEntry) * list.table.size(), s);
}

// The table of launch_apply, which needs one for a single tensor too: without
// it, it takes no offsets.
hipError_t put_snaps(const MxList& list, int32_t nparams, bool stored, void* ws, hipStream_t s,
                     const SnapParam** d_table) {
  char* at = static_cast<char*>(ws) + mx_table_bytes(nparams);
  *d_table = reinterpret_cast<SnapParam*>(at);
  if (stored || nparams == 0) return hipSuccess;
  std::vector<SnapParam> t(static_cast<size_t>(nparams));
  for (int32_t p = 0; p < nparams; ++p) {
    const MxEntry& e = list.table[p];
    t[p] = SnapParam{static_cast<uint16_t*>(e.x), int64_t(e.rows) * e.cols};
  }
  return store_table(at, t.data(), sizeof(SnapParam) * t.size(), s);
}

// Values from which a list's bytes pass through: its 2.5 bytes a value are
// more than the 256 MB that the memory-side cache holds for the next kernel.
constexpr int64_t kStreamElems = int64_t(100) << 20;

template <bool kBack>
void launch_list(const MxEntry* d_table, const MxEntry& one, int32_t nparams, int64_t units,
                 int64_t elems, hipStream_t s) {
  const int span = span_for(units, kMxWantGrid, kBack ? 2 : 4);
  const int grid = grid_for(units, span, kMxMaxGrid);
  if (elems >= kStreamElems)
    mx_list_kernel<kBack, true><<<grid, kMxGroup, 0, s>>>(d_table, one, nparams, units, span);
  else
    mx_list_kernel<kBack, false><<<grid, kMxGroup, 0, s>>>(d_table, one, nparams, units, span);
}

template <bool kBack>
delta_status list_impl(const char* fn, int32_t nparams, void* const* xs, const int32_t* dtypes,
                       const int64_t* rows, const int64_t* cols, uint8_t* const* codes,
                       uint8_t* const* scales, void* ws, size_t ws_bytes, bool stored,
                       hipStream_t s) {
  MxList list;
  delta_status st =
      make_list(fn, nparams, xs, dtypes, rows, cols, codes, scales, kBack, !kBack, stored,
                              &list);
  if (st != DELTA_OK) return st;
  st = check_workspace(fn, ws, ws_bytes, mx_ws_bytes(nparams));
  if (st != DELTA_OK) return st;
  if (list.units == 0) return hip_result(fn, hipSuccess);
  const MxEntry* d_table;
  const hipError_t e = put_table(list, nparams, stored, ws, s, &d_table);
  if (e != hipSuccess) return hip_result(fn, e);
  clear_stale_error();
  launch_list<kBack>(d_table, list.table[0], nparams, list.units, list.elems, s);
  return hip_result(fn, hipGetLastError());
}

// Entries, and values per entry, from where a step takes 1024 of them: then
// groups hold many entries, and a step of 256 has too few groups for its lanes.
// Fewer make small steps, so that a small delta still spreads over the chip.
// us for steps of 256 / 1024: 607M values at 2 % 454 / 491, at 5 % 617 / 589, at
// 9 % 954 / 682; 16.8M values at 5 % 21.0 / 21.4; 1M values at 9 % 7.4 / 11.0.
constexpr int64_t kLargeDelta = int64_t(1) << 20, kLargeSpread = 20;
constexpr int64_t kApplyMaxGrid = int64_t(1) << 20;

template <bool kApply, int kTile>
void launch_apply_tile(const MxEntry* d_table, const MxEntry& one, int32_t nparams,
                       const int32_t* idx, const uint16_t* val, const int64_t* offsets,
                       int64_t max_nnz, hipStream_t s) {
  const int grid = grid_for(max_nnz, kTile, kApplyMaxGrid);
  mx_apply_kernel<kApply, kTile><<<grid, kMxGroup, 0, s>>>(d_table, one, nparams, idx, val,
                                                           offsets, max_nnz);
}

template <bool kApply>
void launch_apply_step(const MxEntry* d_table, const MxEntry& one, int32_t nparams,
                       const int32_t* idx, const uint16_t* val, const int64_t* offsets,
                       int64_t max_nnz, int64_t elems, hipStream_t s) {
  if (max_nnz >= kLargeDelta && max_nnz >= elems / kLargeSpread)
    launch_apply_tile<kApply, 1024>(d_table, one, nparams, idx, val, offsets, max_nnz, s);
  else
    launch_apply_tile<kApply, 256>(d_table, one, nparams, idx, val, offsets, max_nnz, s);
}

// The whole list is quantised as a stream after apply.hip's kernels when there
// is an entry for every kDenseSpread values, and kDenseExtra more, which is
// about what another launch and the list's second pass cost a small list.  us
// for one pass / this: 607M values at 9 % 679 / 718, at 12 % 834 / 731; 16.8M
// at 12 % 27.6 / 30.7, at 20 % 34.0 / 31.9; 1M at 30 % 8.9 / 11.9, at 80 % 16.3 /
// 11.4.
constexpr int64_t kDenseSpread = 10, kDenseExtra = int64_t(1) << 19;

}  // namespace

hipError_t launch_quantize(const void* x, int32_t dtype, int64_t rows, int64_t cols,
                           uint8_t* codes, uint8_t* scales, hipStream_t stream) {
  const int64_t row_blocks = (cols + kMxBlock - 1) / kMxBlock;
  const MxEntry one{const_cast<void*>(x), codes,          scales,
                    0,                    uint32_t(rows), uint32_t(cols),
                    uint32_t(row_blocks), uint32_t(dtype)};
  const int64_t units = (rows * row_blocks + kMxUnit - 1) / kMxUnit;
  clear_stale_error();
  if (units == 0) return hipSuccess;
  launch_list<false>(nullptr, one, 1, units, rows * cols, stream);
  return hipGetLastError();
}

}  // namespace sbd

extern "C" {

size_t mxfp4_workspace_size(int32_t nparams) {
  return nparams < 0 ? 0 : sbd::mx_ws_bytes(nparams);
}

delta_status mxfp4_list_store(int32_t nparams, const void* const* x_ptrs, const int32_t* dtypes,
                              const int64_t* rows, const int64_t* cols, uint8_t* const* code_ptrs,
                              uint8_t* const* scale_ptrs, void* ws, size_t ws_bytes,
                              void* stream) try {
  using namespace sbd;
  const char* fn = "mxfp4_list_store";
  MxList list;
  delta_status st = make_list(fn, nparams, const_cast<void* const*>(x_ptrs), dtypes, rows, cols,
                              code_ptrs, scale_ptrs, true, true, false, &list);
  if (st != DELTA_OK) return st;
  st = check_workspace(fn, ws, ws_bytes, mx_ws_bytes(nparams));
  if (st != DELTA_OK) return st;
  const MxEntry* d_table;
  const SnapParam* d_snaps;
  hipStream_t s = static_cast<hipStream_t>(stream);
  hipError_t e = put_table(list, nparams, false, ws, s, &d_table);
  if (e == hipSuccess) e = put_snaps(list, nparams, false, ws, s, &d_snaps);
  return hip_result(fn, e);
} catch (const std::exception& e) {
  return sbd::fail_with(DELTA_E_INVALID, "mxfp4_list_store: %s", e.what());
}

delta_status mxfp4_quantize_many(int32_t nparams, const void* const* x_ptrs, const int32_t* dtypes,
                                 const int64_t* rows, const int64_t* cols,
                                 uint8_t* const* code_ptrs, uint8_t* const* scale_ptrs, void* ws,
                                 size_t ws_bytes, int32_t table_stored, void* stream) try {
  return sbd::list_impl<false>("mxfp4_quantize_many", nparams, const_cast<void* const*>(x_ptrs),
                               dtypes, rows, cols, code_ptrs, scale_ptrs, ws, ws_bytes,
                               table_stored != 0, static_cast<hipStream_t>(stream));
} catch (const std::exception& e) {
  return sbd::fail_with(DELTA_E_INVALID, "mxfp4_quantize_many: %s", e.what());
}

delta_status mxfp4_dequantize_many(int32_t nparams, const uint8_t* const* code_ptrs,
                                   const uint8_t* const* scale_ptrs, const int64_t* rows,
                                   const int64_t* cols, void* const* x_ptrs, const int32_t* dtypes,
                                   void* ws, size_t ws_bytes, void* stream) try {
  return sbd::list_impl<true>("mxfp4_dequantize_many", nparams, x_ptrs, dtypes, rows, cols,
                              const_cast<uint8_t* const*>(code_ptrs),
                              const_cast<uint8_t* const*>(scale_ptrs), ws, ws_bytes, false,
                              static_cast<hipStream_t>(stream));
} catch (const std::exception& e) {
  return sbd::fail_with(DELTA_E_INVALID, "mxfp4_dequantize_many: %s", e.what());
}

delta_status mxfp4_apply_many(int32_t nparams, uint16_t* const* snap_ptrs, const int64_t* rows,
                              const int64_t* cols, uint8_t* const* code_ptrs,
                              uint8_t* const* scale_ptrs, const int32_t* idx,
                              const uint16_t* val, const int64_t* offsets, int64_t max_nnz,
                              int64_t* violations, void* ws, size_t ws_bytes,
                              int32_t table_stored, void* stream) try {
  using namespace sbd;
  const char* fn = "mxfp4_apply_many";
  if (max_nnz < 0)
    return fail_with(DELTA_E_INVALID, "%s: max_nnz=%lld", fn, (long long)max_nnz);
  if (max_nnz > (int64_t(1) << 62))
    return fail_with(DELTA_E_RANGE, "%s: max_nnz=%lld above 2^62", fn, (long long)max_nnz);
  if (nparams > 0 && max_nnz > 0 && (idx == nullptr || val == nullptr || offsets == nullptr))
    return fail_with(DELTA_E_INVALID, "%s: null idx, val or offsets", fn);
  MxList list;
  const bool stored = table_stored != 0;
  delta_status st = make_list(fn, nparams, reinterpret_cast<void* const*>(snap_ptrs), nullptr,
                              rows, cols, code_ptrs, scale_ptrs, true, true, stored, &list);
  if (st != DELTA_OK) return st;
  st = check_workspace(fn, ws, ws_bytes, mx_ws_bytes(nparams));
  if (st != DELTA_OK) return st;
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (nparams == 0) max_nnz = 0;
  const bool any = list.units > 0 && max_nnz > 0;
  const bool dense = max_nnz >= list.elems / kDenseSpread + kDenseExtra;
  const MxEntry* d_table = nullptr;
  hipError_t e = any ? put_table(list, nparams, stored, ws, s, &d_table) : hipSuccess;
  if (e != hipSuccess) return hip_result(fn, e);
  if (violations != nullptr || (any && dense)) {
    // the counting apply, and the one that is made for dense deltas
    const SnapParam* d_snaps = nullptr;
    if (max_nnz > 0) e = put_snaps(list, nparams, stored, ws, s, &d_snaps);
    if (e == hipSuccess)
      e = launch_apply(d_snaps, SnapParam{nullptr, 0}, nparams, offsets, idx, val, max_nnz,
                       list.elems, violations, s);
    if (e != hipSuccess) return hip_result(fn, e);
  }
  if (!any) return hip_result(fn, hipSuccess);
  clear_stale_error();
  if (dense)
    launch_list<false>(d_table, list.table[0], nparams, list.units, list.elems, s);
  else if (violations != nullptr)
    launch_apply_step<false>(d_table, list.table[0], nparams, idx, val, offsets, max_nnz,
                             list.elems, s);
  else
    launch_apply_step<true>(d_table, list.table[0], nparams, idx, val, offsets, max_nnz,
                            list.elems, s);
  return hip_result(fn, hipGetLastError());
} catch (const std::exception& e) {
  return sbd::fail_with(DELTA_E_INVALID, "mxfp4_apply_many: %s", e.what());
}

}  // extern "C"
