// Activations to 8 bits and back (act8.h): one pass, a thread per 8 channels; memory
// bound.  304,878 x 128 bf16: packed in 20.3 us, unpacked in 19.8 (118 MB each, 5.8 and
// 6.0 TB/s).
#include "act8.h"
#include "launch.h"

namespace ts {

namespace {

template <typename T>
__global__ __launch_bounds__(256) void k_act_pack(const T* __restrict__ x, int64_t units, int per_row, int c, bool vec,
                                                  Act8 a) {
  // units is a multiple of 4, so the 4 lanes of a block stay together
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; i < units; i += int64_t{256} * gridDim.x) {
    const int64_t row = i / per_row;
    const int c0 = static_cast<int>(i - row * per_row) * 8;
    float f[8];
    load_unit(x + row * c, c0, c, vec, f);
    uint32_t byte;
    const ux2 codes = act8_encode(f, &byte);
    act8_store(a, row, c0, c, codes, byte);
  }
}

template <typename T>
__global__ __launch_bounds__(256) void k_act_unpack(Act8 a, int64_t units, int per_row, int c, bool vec,
                                                    T* __restrict__ x) {
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; i < units; i += int64_t{256} * gridDim.x) {
    const int64_t row = i / per_row;
    const int c0 = static_cast<int>(i - row * per_row) * 8;
    float f[8];
    act8_load(a, row, c0, c, f);
    store_unit(x + row * c, c0, c, vec, f);
  }
}

// Blocks for `units` threads: as many as there is work for, below the 2^32
// threads a launch may have (the kernels step over the rest).
unsigned grid_for(int64_t units) {
  const int64_t b = ceil_div<int64_t>(units, 256), most = int64_t{1} << 23;
  return static_cast<unsigned>(b < most ? b : most);
}

template <typename T>
hipError_t pack(const void* x, int64_t n, int c, const Act8& a, hipStream_t s) {
  const int per_row = ceil_div(c, kActBlock) * 4;
  const int64_t units = n * per_row;
  const bool vec = c % 8 == 0 && (reinterpret_cast<uintptr_t>(x) & 15) == 0;
  k_act_pack<T><<<grid_for(units), 256, 0, s>>>(static_cast<const T*>(x), units,
                                                                                     per_row, c, vec, a);
  return hipGetLastError();
}

template <typename T>
hipError_t unpack(const Act8& a, int64_t n, int c, void* x, hipStream_t s) {
  const int per_row = ceil_div(c, 8);
  const int64_t units = n * per_row;
  const bool vec = c % 8 == 0 && (reinterpret_cast<uintptr_t>(x) & 15) == 0;
  k_act_unpack<T><<<grid_for(units), 256, 0, s>>>(a, units, per_row, c, vec,
                                                                                       static_cast<T*>(x));
  return hipGetLastError();
}

}  // namespace

hipError_t launch_act_pack(const void* x, int64_t n, int c, ts_dtype dt, const Act8& a, hipStream_t s) {
  if (n == 0) return hipSuccess;
  switch (dt) {
    case TS_F32: return pack<float>(x, n, c, a, s);
    case TS_F16: return pack<_Float16>(x, n, c, a, s);
    default: return pack<__bf16>(x, n, c, a, s);
  }
}

hipError_t launch_act_unpack(const Act8& a, int64_t n, int c, void* x, ts_dtype dt, hipStream_t s) {
  if (n == 0) return hipSuccess;
  switch (dt) {
    case TS_F32: return unpack<float>(a, n, c, x, s);
    case TS_F16: return unpack<_Float16>(a, n, c, x, s);
    default: return unpack<__bf16>(a, n, c, x, s);
  }
}

}  // namespace ts
