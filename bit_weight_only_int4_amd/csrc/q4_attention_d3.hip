// q4_attention_d3.hip -- attention for 16-bit queries (three digits).
#include "q4_attention_launch.h"

namespace q4 {
template hipError_t launch_attention_digits<3>(const AttnParams& p, hipStream_t s);
}
