// launch.h - a kernel launch that reports its own status.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <tuple>
#include <utility>

namespace km {

// kernel<<<blocks, threads, lds, stream>>>(args...). What is returned is the status of
// this launch. (hipGetLastError after it would also give, and clear, the error that an
// earlier call of this thread has left behind: an in-place kernel that ran would look as
// if it had not.)
template <class... P, size_t... I>
hipError_t launch_with(void (*kernel)(P...), dim3 blocks, dim3 threads, size_t lds,
                       hipStream_t stream, std::tuple<P...> args, std::index_sequence<I...>) {
    void *at[] = {(void *)&std::get<I>(args)...};
    return hipLaunchKernel((const void *)kernel, blocks, threads, at, lds, stream);
}
template <class... P, class... A>
hipError_t launch(void (*kernel)(P...), int64_t blocks, int threads, size_t lds,
                  hipStream_t stream, const A &...args) {
    return launch_with(kernel, dim3((unsigned)blocks), dim3((unsigned)threads), lds, stream,
                       std::tuple<P...>(args...), std::index_sequence_for<P...>{});
}

}  // namespace km
