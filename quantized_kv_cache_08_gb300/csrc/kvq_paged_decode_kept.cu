// The split kernel of kvq_paged_decode.cu for tiles of 8 queries, keeping the
// scores that it works out (launch_split_kept).  A separate translation unit keeps the
// other instances' code unchanged.
#define KVQ_PAGED_KEEP 1
#include "kvq_paged_decode.cu"
