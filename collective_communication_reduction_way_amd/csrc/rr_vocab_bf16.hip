// rr_vocab_bf16.hip -- the vocabulary cross entropy's matrix products, bf16.
#include "rr_vocab_impl.h"

namespace rr {

RR_VOCAB_UNIT(bf16, EBF16)

}  // namespace rr
