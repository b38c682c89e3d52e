// A stand-in for the part of the HIP runtime that the network operators' library calls: launches are
// looked at, not run.  Loaded before the library, in a process of its own.
#include <cstdint>
#include <cstring>
#include <map>
#include <mutex>
#include <utility>

#include <hip/hip_runtime_api.h>

namespace {
std::mutex guard;
int device = 0;
struct Configuration {
    dim3 grid, block;
    size_t lds;
    hipStream_t stream;
} pushed;
std::map<std::pair<int, const void *>, int> allowed;
int64_t launches, blocks, too_many_threads, too_much_lds, attributes;
bool refuse_attributes;
}  // namespace

extern "C" {
hipError_t hipGetDevice(int *id)
{
    *id = device;
    return hipSuccess;
}
hipError_t hipGetLastError() { return hipSuccess; }
hipError_t hipFuncSetAttribute(const void *function, hipFuncAttribute, int value)
{
    std::lock_guard<std::mutex> hold(guard);
    ++attributes;
    if (refuse_attributes)
        return hipErrorInvalidValue;
    allowed[{device, function}] = value;
    return hipSuccess;
}
hipError_t __hipPushCallConfiguration(dim3 grid, dim3 block, size_t lds, hipStream_t stream)
{
    pushed = {grid, block, lds, stream};
    return hipSuccess;
}
hipError_t __hipPopCallConfiguration(dim3 *grid, dim3 *block, size_t *lds, hipStream_t *stream)
{
    *grid = pushed.grid, *block = pushed.block, *lds = pushed.lds, *stream = pushed.stream;
    return hipSuccess;
}
hipError_t hipLaunchKernel(const void *function, dim3 grid, dim3 block, void **, size_t lds, hipStream_t)
{
    std::lock_guard<std::mutex> hold(guard);
    ++launches;
    blocks += (int64_t)grid.x * grid.y;
    // threads are counted in 32 bits along each axis
    if ((uint64_t)grid.x * block.x > 0xffffffffull || (uint64_t)grid.y * block.y > 0xffffffffull || grid.y > 65535)
        ++too_many_threads;
    if (lds > 64 * 1024) {
        const auto at = allowed.find({device, function});
        if (at == allowed.end() || (size_t)at->second < lds)
            ++too_much_lds;
    }
    return hipSuccess;
}

void stand_in_device(int id) { device = id; }
void stand_in_refuses(int yes) { refuse_attributes = yes != 0; }
// launches, blocks, launches of too many threads, launches of more LDS than allowed, calls that allow it
void stand_in_counts(int64_t *out)
{
    const int64_t all[] = {launches, blocks, too_many_threads, too_much_lds, attributes};
    std::memcpy(out, all, sizeof(all));
}
}
