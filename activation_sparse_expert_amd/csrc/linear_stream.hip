// Linear layer on 16-bit types, streamed.
#include "linear_stream.hpp"

namespace moeffn {

hipError_t launch_linear_stream(const LinearArgs &a, hipStream_t s)
{
    return a.bf16 ? launch_stream<st::kBF16>(a, s) : launch_stream<st::kF16>(a, s);
}

}  // namespace moeffn
