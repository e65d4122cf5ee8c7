"""Small programs that run the library's calls together as a user would."""
