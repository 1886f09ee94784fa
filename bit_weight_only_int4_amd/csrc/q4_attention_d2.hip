// q4_attention_d2.hip -- attention for 16-bit queries (two digits).
#include "q4_attention_launch.h"

namespace q4 {
template hipError_t launch_attention_digits<2>(const AttnParams& p, hipStream_t s);
}
